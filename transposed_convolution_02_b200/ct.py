"""Python binding of libct.so (include/ct.h): argument marshalling only.

The functions carry the C names (``ct_output_shape``, ``ct_plan``,
``ct_prepack_weights``, ``ct_run`` ...) and take plain integers for device
pointers and streams.  ``ConvTranspose`` wraps them for torch tensors: torch
provides the device memory and the stream, every step of the operator runs
in the library's CUDA kernels.  There is no fallback: when libct.so is
missing or the device is not an sm_100 part, calls raise.

Attribute names follow the ai.onnx.ConvTranspose README ("Attributes");
``conv_transpose_nhwc`` follows ClikaRT::ops::conv_transpose (channels-last,
weight [C_in, K.., O/groups], padding as (lo, hi) per spatial dim).
"""

import array
import ctypes
import functools
import math
import numbers
import os

import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libct.so")

CT_OK = 0
STATUS_NAMES = {0: "CT_OK", 1: "CT_ERR_CHANNELS", 2: "CT_ERR_SPAN", 3: "CT_ERR_DTYPE",
                4: "CT_ERR_ATTR", 5: "CT_ERR_ALIGN", 6: "CT_ERR_NULL", 7: "CT_ERR_DEVICE",
                8: "CT_ERR_WORKSPACE", 9: "CT_ERR_UNSUPPORTED", 10: "CT_ERR_NOMEM"}
CT_F32, CT_F16, CT_BF16 = 0, 1, 2
CT_NCHW, CT_NHWC = 0, 1
AUTOPAD = {"NOTSET": 0, "SAME_UPPER": 1, "SAME_LOWER": 2, "VALID": 3}
ALGO = {"auto": 0, "generic": 1, "dense_tc": 2, "fp32_gemm": 3, "grouped": 4,
        "dense_tc_pertap": 5, "dense_tc_pair": 6}

PART_PREPARE, PART_MAIN, PART_ALL = 1, 2, 3

EXPORTED = ["ct_output_shape", "ct_plan", "ct_plan_kernel", "ct_plan_launches",
            "ct_prepacked_weight_bytes",
            "ct_workspace_bytes", "ct_prepack_weights", "ct_run", "ct_run_parts",
            "ct_run_noalloc", "ct_plan_destroy", "ct_status_string", "ct_take_device_error",
            "ct_selftest_wait_timeout", "ct_dropout", "ct_group_norm", "ct_group_norm_backward",
            "ct_group_norm_workspace_bytes", "ct_rms_norm", "ct_rms_norm_e4m3",
            "ct_rms_norm_backward", "ct_rms_norm_workspace_bytes", "ct_rotary",
            "ct_adamw", "ct_grad_norm", "ct_grad_norm_workspace_bytes"]


class CtError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS_NAMES.get(status, status),
                                          ct_status_string(status)))


class ct_desc(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("auto_pad", ctypes.c_int32),
                ("N", ctypes.c_int64), ("C", ctypes.c_int64),
                ("in_", ctypes.c_int64 * 3), ("w_dims", ctypes.c_int64 * 5),
                ("group", ctypes.c_int64), ("bias_len", ctypes.c_int64),
                ("strides", ctypes.c_int64 * 3), ("dilations", ctypes.c_int64 * 3),
                ("pads", ctypes.c_int64 * 6), ("output_padding", ctypes.c_int64 * 3),
                ("has_kernel_shape", ctypes.c_int32), ("has_output_shape", ctypes.c_int32),
                ("kernel_shape", ctypes.c_int64 * 3), ("output_shape", ctypes.c_int64 * 3),
                ("algo", ctypes.c_int32), ("activation", ctypes.c_int32)]


class ct_group_norm_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("N", ctypes.c_int64), ("S", ctypes.c_int64), ("C", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("eps", ctypes.c_double)]


class ct_rms_norm_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("block", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("C", ctypes.c_int64), ("eps", ctypes.c_double)]


class ct_rotary_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("axes", ctypes.c_int32), ("pairs", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("position_type", ctypes.c_int32),
                ("position_images", ctypes.c_int32), ("N", ctypes.c_int64),
                ("grid", ctypes.c_int64 * 3), ("heads", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("sections", ctypes.c_int64 * 3), ("x_strides", ctypes.c_int64 * 3),
                ("y_strides", ctypes.c_int64 * 3), ("base", ctypes.c_double)]


class ct_param(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("weight_decay", ctypes.c_double)]


class ct_adamw_desc(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("reserved", ctypes.c_int32), ("lr", ctypes.c_double),
                ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("lr_device", ctypes.c_void_p),
                ("step_device", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libct.so (raises when it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libct.so is not built (%s); run "
                              "transposed_convolution_02_b200/build.py" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        i64p = ctypes.POINTER(ctypes.c_int64)
        szp = ctypes.POINTER(ctypes.c_size_t)
        dp = ctypes.POINTER(ct_desc)
        L.ct_output_shape.argtypes = [dp, i64p, i64p, i64p]
        L.ct_plan.argtypes = [dp, ctypes.POINTER(P)]
        L.ct_plan_kernel.argtypes = [P]
        L.ct_plan_kernel.restype = ctypes.c_char_p
        L.ct_plan_launches.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        L.ct_prepacked_weight_bytes.argtypes = [P, szp]
        L.ct_workspace_bytes.argtypes = [P, szp]
        L.ct_prepack_weights.argtypes = [P, P, P, P]
        L.ct_run.argtypes = [P, P, P, P, P, P, P]
        L.ct_run_parts.argtypes = [P, P, P, P, P, P, P, ctypes.c_int32]
        L.ct_selftest_wait_timeout.argtypes = [P, ctypes.c_int64]
        L.ct_run_noalloc.argtypes = [P, P, P, P, P, P]
        L.ct_plan_destroy.argtypes = [P]
        L.ct_plan_destroy.restype = None
        L.ct_take_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        gp, u64, f64 = ctypes.POINTER(ct_group_norm_desc), ctypes.c_uint64, ctypes.c_double
        L.ct_dropout.argtypes = [ctypes.c_int32, ctypes.c_int64, P, P, f64, u64, u64, P, P, P]
        L.ct_group_norm_workspace_bytes.argtypes = [gp, szp, szp]
        L.ct_group_norm.argtypes = [gp, P, P, P, f64, u64, u64, P, P, P, P, P, P]
        L.ct_group_norm_backward.argtypes = [gp, P, P, P, P, P, P, f64, u64, u64, P, P, P, P, P, P]
        rp = ctypes.POINTER(ct_rms_norm_desc)
        L.ct_rms_norm_workspace_bytes.argtypes = [rp, szp]
        L.ct_rms_norm.argtypes = [rp, P, P, P, P, P, P, P]
        L.ct_rms_norm_e4m3.argtypes = [rp, P, P, P, P, P, P, P, P]
        L.ct_rms_norm_backward.argtypes = [rp, P, P, P, P, P, P, P, P, P]
        L.ct_rotary.argtypes = [ctypes.POINTER(ct_rotary_desc), P, P, P, P]
        L.ct_adamw.argtypes = [ctypes.POINTER(ct_adamw_desc), ctypes.c_int64, ctypes.POINTER(ct_param),
                               P, P, P, P, P, P, P, P]
        L.ct_grad_norm_workspace_bytes.argtypes = [ctypes.c_int64, szp]
        L.ct_grad_norm.argtypes = [ctypes.c_int64, ctypes.POINTER(ct_param), P, f64, P, P, P, P]
        L.ct_status_string.argtypes = [ctypes.c_int]
        L.ct_status_string.restype = ctypes.c_char_p
        for name in ("ct_output_shape", "ct_plan", "ct_plan_launches", "ct_prepacked_weight_bytes",
                     "ct_workspace_bytes", "ct_prepack_weights", "ct_run", "ct_run_parts",
                     "ct_run_noalloc", "ct_take_device_error", "ct_selftest_wait_timeout",
                     "ct_dropout", "ct_group_norm", "ct_group_norm_backward",
                     "ct_group_norm_workspace_bytes", "ct_rms_norm", "ct_rms_norm_e4m3",
                     "ct_rms_norm_backward", "ct_rms_norm_workspace_bytes", "ct_rotary",
                     "ct_adamw", "ct_grad_norm", "ct_grad_norm_workspace_bytes"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


# ---- the C entry points, same names -------------------------------------

def ct_status_string(status):
    return lib().ct_status_string(int(status)).decode()


def ct_output_shape(desc):
    y = (ctypes.c_int64 * 5)()
    pb = (ctypes.c_int64 * 3)()
    pe = (ctypes.c_int64 * 3)()
    st = lib().ct_output_shape(ctypes.byref(desc), y, pb, pe)
    if st != CT_OK:
        raise CtError(st, "ct_output_shape")
    r = desc.rank
    return list(y)[: r + 2], list(pb)[:r], list(pe)[:r]


def ct_plan(desc):
    h = ctypes.c_void_p()
    st = lib().ct_plan(ctypes.byref(desc), ctypes.byref(h))
    if st != CT_OK:
        raise CtError(st, "ct_plan")
    return h


def ct_plan_kernel(plan):
    return lib().ct_plan_kernel(plan).decode()


def ct_plan_launches(plan):
    n = ctypes.c_int32()
    st = lib().ct_plan_launches(plan, ctypes.byref(n))
    if st != CT_OK:
        raise CtError(st, "ct_plan_launches")
    return n.value


def ct_prepacked_weight_bytes(plan):
    n = ctypes.c_size_t()
    st = lib().ct_prepacked_weight_bytes(plan, ctypes.byref(n))
    if st != CT_OK:
        raise CtError(st, "ct_prepacked_weight_bytes")
    return n.value


def ct_workspace_bytes(plan):
    n = ctypes.c_size_t()
    st = lib().ct_workspace_bytes(plan, ctypes.byref(n))
    if st != CT_OK:
        raise CtError(st, "ct_workspace_bytes")
    return n.value


def ct_prepack_weights(plan, w_ptr, wp_ptr, stream):
    st = lib().ct_prepack_weights(plan, w_ptr, wp_ptr, stream)
    if st != CT_OK:
        raise CtError(st, "ct_prepack_weights")


def ct_run(plan, x_ptr, wp_ptr, bias_ptr, y_ptr, ws_ptr, stream):
    st = lib().ct_run(plan, x_ptr, wp_ptr, bias_ptr, y_ptr, ws_ptr, stream)
    if st != CT_OK:
        raise CtError(st, "ct_run")


def ct_run_parts(plan, x_ptr, wp_ptr, bias_ptr, y_ptr, ws_ptr, stream, parts):
    """ct_run restricted to a mask of PART_PREPARE (re-layout, bias fill) and
    PART_MAIN (the main kernel), for timing the parts of a call apart."""
    st = lib().ct_run_parts(plan, x_ptr, wp_ptr, bias_ptr, y_ptr, ws_ptr, stream, int(parts))
    if st != CT_OK:
        raise CtError(st, "ct_run_parts")


def ct_selftest_wait_timeout(limit_cycles, stream=None):
    """Launch the bounded-wait self-test (a wait that gives up after
    `limit_cycles` SM cycles, then drains its copy in flight); the next
    ct_take_device_error() returns 501."""
    st = lib().ct_selftest_wait_timeout(_stream_ptr(stream), int(limit_cycles))
    if st != CT_OK:
        raise CtError(st, "ct_selftest_wait_timeout")


def ct_run_noalloc(plan, x_ptr, wp_ptr, bias_ptr, y_ptr, stream):
    """ct_run with the workspace taken from the library's fixed device array
    (for callers that may not allocate device memory while running)."""
    st = lib().ct_run_noalloc(plan, x_ptr, wp_ptr, bias_ptr, y_ptr, stream)
    if st != CT_OK:
        raise CtError(st, "ct_run_noalloc")


def ct_take_device_error(stream=None):
    """Wait for the stream, then read and clear the kernels' device error
    words: 0 when no bounded wait ran out since the last call, else the code
    100 * module + wait site.  Raises CtError when a CUDA call failed."""
    code = ctypes.c_int32()
    st = lib().ct_take_device_error(_stream_ptr(stream) if torch.cuda.is_available() else None,
                                    ctypes.byref(code))
    if st != CT_OK and code.value == 0:
        raise CtError(st, "ct_take_device_error")
    return code.value


def ct_plan_destroy(plan):
    if plan:
        lib().ct_plan_destroy(plan)


# ---- descriptor construction ----------------------------------------------

ACTIVATION = {"identity": 0, "relu": 1}
NORM_ACTIVATION = {"identity": 0, "relu": 1, "silu": 2, "gelu": 3}
NORM_DTYPE = {torch.float32: CT_F32, torch.float16: CT_F16, torch.bfloat16: CT_BF16}


def make_desc(x_shape, w_shape, *, dtype, layout="nchw", strides=None, dilations=None,
              pads=None, output_padding=None, auto_pad="NOTSET", group=1, bias_len=0,
              kernel_shape=None, output_shape=None, algo="auto", activation="identity"):
    """Fill a ct_desc from tensor shapes and README-named attributes."""
    d = ct_desc()
    r = len(x_shape) - 2
    d.rank = r
    d.dtype = {torch.float32: CT_F32, torch.float16: CT_F16}.get(dtype, 99)
    d.layout = CT_NCHW if layout == "nchw" else CT_NHWC
    d.auto_pad = AUTOPAD.get(auto_pad, 99)
    d.N = int(x_shape[0])
    if layout == "nchw":
        d.C = int(x_shape[1])
        sp = x_shape[2:]
    else:
        d.C = int(x_shape[-1])
        sp = x_shape[1:-1]
    for a in range(min(r, 3)):
        d.in_[a] = int(sp[a])
    for a, v in enumerate(list(w_shape)[:5]):
        d.w_dims[a] = int(v)
    d.group = int(group)
    d.bias_len = int(bias_len)
    for a in range(min(r, 3)):
        d.strides[a] = int(strides[a]) if strides is not None else 1
        d.dilations[a] = int(dilations[a]) if dilations is not None else 1
        d.output_padding[a] = int(output_padding[a]) if output_padding is not None else 0
    if pads is not None:
        for a, v in enumerate(list(pads)[:6]):
            d.pads[a] = int(v)
    if kernel_shape is not None:
        d.has_kernel_shape = 1
        for a, v in enumerate(list(kernel_shape)[:3]):
            d.kernel_shape[a] = int(v)
    if output_shape is not None:
        d.has_output_shape = 1
        for a, v in enumerate(list(output_shape)[:3]):
            d.output_shape[a] = int(v)
    d.algo = ALGO[algo]
    d.activation = ACTIVATION.get(activation, 99)
    return d


# ---- torch-facing wrapper ---------------------------------------------------

def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def check_io(x, out, x_shape, y_shape, dtype, device):
    """Refuse a call whose tensors do not match the plan (the kernels trust the
    planned sizes: a different X or Y would be read or written out of bounds)."""
    if list(x.shape) != list(x_shape):
        raise ValueError("X has shape %s, the plan was made for %s" % (list(x.shape), list(x_shape)))
    if x.dtype != dtype:
        raise ValueError("X is %s, the plan computes in %s" % (x.dtype, dtype))
    if x.device != device:
        raise ValueError("X is on %s, the packed weights on %s" % (x.device, device))
    if out is not None:
        if list(out.shape) != list(y_shape) or out.dtype != dtype or out.device != device:
            raise ValueError("out must be a %s tensor of shape %s on %s" % (dtype, list(y_shape), device))
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")


class ConvTranspose:
    """A planned ConvTranspose with its weight pre-packed on the device.

    Plan and pre-pack happen once here; ``__call__`` allocates Y (and the
    workspace once) with torch and launches ``ct_run`` on the current stream.
    """

    def __init__(self, w, x_shape, bias=None, *, layout="nchw", strides=None, dilations=None,
                 pads=None, output_padding=None, auto_pad="NOTSET", group=1,
                 kernel_shape=None, output_shape=None, algo="auto", activation="identity",
                 stream=None):
        if not w.is_cuda:
            raise ValueError("W must be a CUDA tensor")
        if bias is not None and (bias.dtype != w.dtype or bias.device != w.device):
            raise ValueError("bias must be a tensor of W's dtype on W's device")
        self.layout = layout
        self.dtype = w.dtype
        self.device = w.device
        self.x_shape = list(x_shape)
        self.desc = make_desc(list(x_shape), list(w.shape), dtype=w.dtype, layout=layout,
                              strides=strides, dilations=dilations, pads=pads,
                              output_padding=output_padding, auto_pad=auto_pad, group=group,
                              bias_len=0 if bias is None else bias.numel(),
                              kernel_shape=kernel_shape, output_shape=output_shape, algo=algo,
                              activation=activation)
        self.y_shape, self.pad_begin, self.pad_end = ct_output_shape(self.desc)
        self.plan = ct_plan(self.desc)
        self.kernel = ct_plan_kernel(self.plan)
        self.launches = ct_plan_launches(self.plan)
        nb = ct_prepacked_weight_bytes(self.plan)
        self.w_packed = torch.empty(max(nb, 16), dtype=torch.uint8, device=w.device)
        ws = ct_workspace_bytes(self.plan)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=w.device) if ws else None
        self.bias = bias.contiguous() if bias is not None else None
        w = w.contiguous()
        ct_prepack_weights(self.plan, _ptr(w), _ptr(self.w_packed), _stream_ptr(stream))
        self._w_keep = w

    def __call__(self, x, out=None, stream=None):
        if not x.is_cuda:
            raise ValueError("X must be a CUDA tensor")
        check_io(x, out, self.x_shape, self.y_shape, self.dtype, self.device)
        x = x.contiguous()
        y = out if out is not None else torch.empty(self.y_shape, dtype=self.dtype,
                                                    device=x.device)
        ct_run(self.plan, _ptr(x), _ptr(self.w_packed), _ptr(self.bias), _ptr(y),
               _ptr(self.workspace), _stream_ptr(stream))
        return y

    def run_ptrs(self, x_ptr, y_ptr, stream_ptr, parts=PART_ALL):
        """Launch on raw device pointers (benchmark loops); the caller
        guarantees buffers of the planned shapes, dtype and device.  `parts`
        restricts the call to its preparation or main launches."""
        ct_run_parts(self.plan, x_ptr, _ptr(self.w_packed), _ptr(self.bias), y_ptr,
                     _ptr(self.workspace), stream_ptr, parts)

    def run_part(self, x, out, parts, stream=None):
        """ct_run_parts on tensors checked against the plan (see run_ptrs)."""
        check_io(x, out, self.x_shape, self.y_shape, self.dtype, self.device)
        if out is None or not x.is_contiguous():
            raise ValueError("run_part needs a contiguous X and an out tensor")
        ct_run_parts(self.plan, _ptr(x), _ptr(self.w_packed), _ptr(self.bias), _ptr(out),
                     _ptr(self.workspace), _stream_ptr(stream), parts)
        return out

    def __del__(self):
        try:
            ct_plan_destroy(self.plan)
        except Exception:
            pass


def conv_transpose(x, w, bias=None, *, strides=None, dilations=None, pads=None,
                   output_padding=None, auto_pad="NOTSET", group=1, kernel_shape=None,
                   output_shape=None, algo="auto", activation="identity"):
    """ONNX ConvTranspose, channels-first: X[N,C,D..], W[C,M/group,k..] -> Y
    (optionally followed by the activation, identity by default)."""
    op = ConvTranspose(w, list(x.shape), bias, layout="nchw", strides=strides,
                       dilations=dilations, pads=pads, output_padding=output_padding,
                       auto_pad=auto_pad, group=group, kernel_shape=kernel_shape,
                       output_shape=output_shape, algo=algo, activation=activation)
    return op(x)


def conv_transpose_nhwc(x, w, bias=None, *, stride, padding, output_padding, groups,
                        dilation, activation="identity", algo="auto"):
    """Channels-last call in the form of ClikaRT::ops::conv_transpose: input
    [N, D.., C_in], weight [C_in, K.., O/groups], padding (lo, hi) per spatial
    dim, activation (identity or relu), output [N, out.., C_out]."""
    r = x.dim() - 2
    if len(padding) != 2 * r:
        raise ValueError("padding needs two entries (lo, hi) per spatial dim")
    pads = [padding[2 * a] for a in range(r)] + [padding[2 * a + 1] for a in range(r)]
    op = ConvTranspose(w, list(x.shape), bias, layout="nhwc", strides=stride,
                       dilations=dilation, pads=pads, output_padding=output_padding,
                       group=groups, algo=algo, activation=activation)
    return op(x)


# ---- group norm and dropout ---------------------------------------------------

def _overlap(a, b):
    """Whether two contiguous tensors share memory."""
    a0, b0 = a.data_ptr(), b.data_ptr()
    return (a0 < b0 + b.numel() * b.element_size() and b0 < a0 + a.numel() * a.element_size())


def check_like(t, name, x):
    """Refuse a tensor that has not X's shape, dtype and device."""
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError("%s must be a %s tensor of shape %s on %s"
                         % (name, x.dtype, list(x.shape), x.device))


def check_out(out, x, inputs, in_place=False):
    """Refuse an output that the kernels could not fill: not like X, not dense,
    or over an input (`in_place`: exactly on one of them is fine)."""
    check_like(out, "out", x)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    for t in inputs:
        if t is not None and _overlap(out, t) and not (in_place and out.data_ptr() == t.data_ptr()
                                                       and t.is_contiguous()):
            raise ValueError("out overlaps an input")


def check_random(p, seed, offset, rng, device):
    """Refuse a drop probability outside [0, 1], a seed or offset outside
    64 bits, and an rng that is not two int64 words on X's device."""
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1]")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be in [0, 2^64)")
    if rng is not None and (rng.dtype != torch.int64 or rng.device != device or rng.dim() != 1
                            or rng.numel() != 2 or not rng.is_contiguous()):
        raise ValueError("rng must be an int64 tensor [seed, offset] on %s" % (device,))


def check_norm(x, groups, weight, bias, activation):
    """Refuse arguments that the group norm cannot take."""
    if x.dtype not in NORM_DTYPE:
        raise ValueError("X must be float32, float16 or bfloat16, not %s" % x.dtype)
    if x.dim() < 2:
        raise ValueError("X must be [N, D.., C], it has shape %s" % list(x.shape))
    c = x.shape[-1]
    if groups < 1 or groups % 1 != 0 or c < 1 or c % groups != 0:
        raise ValueError("%d channels cannot be split into %s groups" % (c, groups))
    if activation not in NORM_ACTIVATION:
        raise ValueError("activation must be one of %s, not %r" % (sorted(NORM_ACTIVATION), activation))
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if t.dtype != torch.float32 and t.dtype != x.dtype:
            raise ValueError("%s must be float32 or X's %s, not %s" % (name, x.dtype, t.dtype))
        if t.dim() != 1 or t.numel() != c or t.device != x.device:
            raise ValueError("%s must have shape [%d] on %s" % (name, c, x.device))
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")


def _check_cuda(x, *leaves):
    """The operators run on CUDA tensors only and record no derivatives: a call
    that would drop a gradient or a forward-mode tangent silently is refused."""
    if not x.is_cuda:
        raise ValueError("X must be a CUDA tensor")
    if forward_ad._current_level >= 0:      # within a dual_level, whatever the grad mode
        for t in (x,) + leaves:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("an input or an output carries a forward-mode tangent, and this call computes none")
    if not torch.is_grad_enabled():
        return
    for t in (x,) + leaves:
        if t is None or not t.requires_grad:
            continue
        raise ValueError("an input or an output requires a gradient, and this call records none: call it under "
                         "torch.no_grad() and use the _backward function")


def _elsewhere(call, x, stream):
    """`call(raw stream)` where tensors are allocated and kernels launched for
    X: on its device, on the given stream (the device's current one by
    default)."""
    dev = x.device
    if stream is not None and stream.device != dev:
        raise ValueError("the stream is on %s, X on %s" % (stream.device, dev))
    with torch.cuda.device(dev):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _run_on(call, x, stream):
    index = x.get_device()
    if stream is None and index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(index))
    return _elsewhere(call, x, stream)


def _addr(t):
    return None if t is None else t.data_ptr()


def _kept_by_value(*settings):
    """Whether numbers can stand in a key: a tensor would be found by what it is, whatever it holds by then."""
    return all(isinstance(v, numbers.Real) for v in settings)


def _written(*outs):
    """Tell autograd that these tensors of the caller's were overwritten: what saved one of them for its backward
    pass is then refused there."""
    torch.autograd.graph.increment_version([t for t in outs if t is not None])


class _Norm:
    """A group norm's descriptor and workspace sizes: sizes only, no memory."""

    def __init__(self, shape, dtype, groups, param_dtype, activation, eps):
        s = 1
        for v in shape[1:-1]:
            s *= v
        self.shape, self.dtype = shape, dtype
        self.stats = (shape[0], groups)
        self.desc = ct_group_norm_desc(NORM_DTYPE[dtype], NORM_DTYPE[param_dtype],
                                       NORM_ACTIVATION[activation], 0, shape[0], s, shape[-1], groups, eps)
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        st = lib().ct_group_norm_workspace_bytes(ctypes.byref(self.desc), ctypes.byref(f), ctypes.byref(b))
        if st != CT_OK:
            raise CtError(st, "ct_group_norm_workspace_bytes")
        self.forward_bytes, self.backward_bytes = f.value, b.value


_norm = functools.lru_cache(maxsize=1024)(_Norm)


def _norm_of(x, groups, weight, bias, activation, eps):
    """The checked arguments' _Norm (the checks by size and type are made once
    per size and type)."""
    one = weight if weight is not None else bias
    pd = torch.float32 if one is None else one.dtype
    try:
        n = _NORMS[x.shape, x.dtype, groups, pd, activation, eps]
    except (KeyError, TypeError):
        check_norm(x, groups, weight, bias, activation)
        n = _norm(x.shape, x.dtype, int(groups), pd, activation, float(eps))
        if _kept_by_value(groups, eps):
            if len(_NORMS) >= 1024:
                _NORMS.clear()
            _NORMS[x.shape, x.dtype, groups, pd, activation, eps] = n
        return n
    dev = x.device
    for t in (weight, bias):
        if t is not None and (t.dtype != pd or t.device != dev or t.dim() != 1 or t.numel() != n.shape[-1]):
            check_norm(x, groups, weight, bias, activation)
    return n


_NORMS = {}


def group_norm_nhwc(x, groups, weight=None, bias=None, *, eps=1e-5, activation="identity", p=0.0,
                    seed=0, offset=0, rng=None, out=None, return_stats=False, stream=None):
    """Group norm of channels-last X[N, D.., C] (what conv_transpose_nhwc
    returns), then the activation (identity, relu, silu or gelu), then dropout
    with probability p (see dropout for seed, offset and rng): float32,
    float16 or bfloat16, weight and bias [C] in X's dtype or float32.  Inputs
    that are not contiguous (a permuted channels-first X) are copied first.
    ``out`` may not overlap an input.

    Returns Y, or (Y, mean, rstd) with ``return_stats``: mean and rstd are
    float32 [N, groups], what group_norm_nhwc_backward takes."""
    norm = _norm_of(x, groups, weight, bias, activation, eps)
    if p:
        check_random(p, seed, offset, rng, x.device)
    if out is not None:
        check_out(out, x, (x, weight, bias, rng if p else None))
    _check_cuda(x, weight, bias, out)

    def call(raw):
        xc = x.contiguous()
        w = None if weight is None else weight.contiguous()
        b = None if bias is None else bias.contiguous()
        y = torch.empty_like(xc) if out is None else out
        if return_stats:
            n, g = norm.stats
            mean, rstd = torch.empty_strided((2, n, g), (n * g, g, 1), dtype=torch.float32,
                                             device=xc.device).unbind()
        else:
            mean = rstd = None
        ws = (torch.empty(norm.forward_bytes, dtype=torch.uint8, device=xc.device) if norm.forward_bytes
              else None)
        st = lib().ct_group_norm(norm.desc, xc.data_ptr(), _addr(w), _addr(b), p, seed, offset,
                                 _addr(rng), y.data_ptr(), _addr(mean), _addr(rstd), _addr(ws), raw)
        if st != CT_OK:
            raise CtError(st, "ct_group_norm")
        if out is not None:
            _written(out)
        return (y, mean, rstd) if return_stats else y

    return _run_on(call, x, stream)


def group_norm_nhwc_backward(dy, x, mean, rstd, groups, weight=None, bias=None, *, activation="identity",
                             p=0.0, seed=0, offset=0, rng=None, need_x_grad=True, stream=None):
    """Gradients (dx, dweight, dbias) of group_norm_nhwc at dy, from the X,
    mean and rstd, the weight and bias and the p, seed, offset and rng of the
    forward call.  None for dx without ``need_x_grad``, and for the gradient
    of a weight or bias that is None."""
    norm = _norm_of(x, groups, weight, bias, activation, 0.0)
    check_like(dy, "dy", x)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.shape != norm.stats or t.device != x.device:
            raise ValueError("%s must be a float32 tensor of shape %s on %s"
                             % (name, list(norm.stats), x.device))
    if p:
        check_random(p, seed, offset, rng, x.device)
    _check_cuda(x, dy, mean, rstd, weight, bias)

    def call(raw):
        xc, dyc, m, r = x.contiguous(), dy.contiguous(), mean.contiguous(), rstd.contiguous()
        w = None if weight is None else weight.contiguous()
        b = None if bias is None else bias.contiguous()
        dx = torch.empty_like(xc) if need_x_grad else None
        dweight = None if w is None else torch.empty_like(w)
        dbias = None if b is None else torch.empty_like(b)
        ws = (torch.empty(norm.backward_bytes, dtype=torch.uint8, device=xc.device)
              if norm.backward_bytes else None)
        st = lib().ct_group_norm_backward(norm.desc, dyc.data_ptr(), xc.data_ptr(), m.data_ptr(),
                                          r.data_ptr(), _addr(w), _addr(b), p, seed, offset, _addr(rng),
                                          _addr(dx), _addr(dweight), _addr(dbias), _addr(ws), raw)
        if st != CT_OK:
            raise CtError(st, "ct_group_norm_backward")
        return dx, dweight, dbias

    return _run_on(call, x, stream)


def dropout(x, p, *, seed=0, offset=0, rng=None, residual=None, out=None, stream=None):
    """Dropout of X with probability p (in steps of 2^-16), plus an optional
    residual: kept elements are scaled so that the expectation is X.

    Which elements stay is a function of their index, seed and offset alone
    (Philox4x32-10), so no mask is stored: give dropout_backward the same
    numbers.  ``rng``, an int64 CUDA tensor [seed, offset], is read on the
    device in their place: a captured graph then draws a new mask at each
    replay once the tensor is changed.  ``out`` may be X or the residual."""
    if x.dtype not in NORM_DTYPE:
        raise ValueError("X must be float32, float16 or bfloat16, not %s" % x.dtype)
    check_random(p, seed, offset, rng, x.device)
    if residual is not None:
        check_like(residual, "residual", x)
    if out is not None:
        check_out(out, x, (x, residual), in_place=True)
        check_out(out, x, (rng,))
    _check_cuda(x, residual, out)

    def call(raw):
        xc = x.contiguous()
        r = None if residual is None else residual.contiguous()
        y = torch.empty_like(xc) if out is None else out
        st = lib().ct_dropout(NORM_DTYPE[xc.dtype], xc.numel(), xc.data_ptr(), _addr(r), p, seed, offset,
                              _addr(rng), y.data_ptr(), raw)
        if st != CT_OK:
            raise CtError(st, "ct_dropout")
        if out is not None:
            _written(out)
        return y

    return _run_on(call, x, stream)


def dropout_backward(dy, p, *, seed=0, offset=0, rng=None, out=None, stream=None):
    """The gradient of dropout in X at dy, for the p, seed, offset and rng of
    the forward call (the residual's gradient is dy itself)."""
    return dropout(dy, p, seed=seed, offset=offset, rng=rng, out=out, stream=stream)


# ---- root-mean-square norm ----------------------------------------------------

class _Rms:
    """A root-mean-square norm's descriptor and workspace size."""

    def __init__(self, shape, dtype, param_dtype, block, eps):
        block = int(block)
        self.rows_shape, self.c = shape[:-1], shape[-1]
        self.scale_shape = self.rows_shape + (-(-self.c // block),) if block else self.rows_shape
        self.desc = ct_rms_norm_desc(NORM_DTYPE[dtype], NORM_DTYPE[param_dtype], block, 0,
                                     math.prod(self.rows_shape), self.c, eps)
        b = ctypes.c_size_t()
        st = lib().ct_rms_norm_workspace_bytes(ctypes.byref(self.desc), ctypes.byref(b))
        if st != CT_OK:
            raise CtError(st, "ct_rms_norm_workspace_bytes")
        self.backward_bytes = b.value


_RMS = {}


def check_rms(x, weight, block):
    """Refuse arguments that the root-mean-square norm cannot take."""
    if x.dtype not in NORM_DTYPE:
        raise ValueError("X must be float32, float16 or bfloat16, not %s" % x.dtype)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("X must be [.., C] with C >= 1, it has shape %s" % list(x.shape))
    if block not in (0, 32, 64, 128):
        raise ValueError("block must be None, 32, 64 or 128, not %r" % (block,))
    if weight is not None:
        if weight.dtype != torch.float32 and weight.dtype != x.dtype:
            raise ValueError("weight must be float32 or X's %s, not %s" % (x.dtype, weight.dtype))
        if weight.dim() != 1 or weight.numel() != x.shape[-1] or weight.device != x.device:
            raise ValueError("weight must have shape [%d] on %s" % (x.shape[-1], x.device))


def _rms_of(x, weight, block, eps):
    """The checked arguments' _Rms (made once per size and type)."""
    pd = torch.float32 if weight is None else weight.dtype
    key = (x.shape, x.dtype, pd, block, eps)
    try:
        r = _RMS[key]
    except (KeyError, TypeError):
        check_rms(x, weight, block)
        r = _Rms(tuple(x.shape), x.dtype, pd, block, float(eps))
        if _kept_by_value(eps, block):
            if len(_RMS) >= 1024:
                _RMS.clear()
            _RMS[key] = r
        return r
    if weight is not None and (weight.dim() != 1 or weight.numel() != r.c or weight.get_device() != x.get_device()):
        check_rms(x, weight, block)
    return r


def _rms_inputs(x, weight, residual, *outs):
    """Checks of both forward calls; `outs` may be X or the residual."""
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype
                                 or residual.get_device() != x.get_device()):
        check_like(residual, "residual", x)
    for t in outs:
        if t is not None:
            check_out(t, x, (x, residual), in_place=True)
            check_out(t, x, (weight,))
    if len(outs) == 2 and outs[0] is not None and outs[1] is not None and _overlap(*outs):
        raise ValueError("out and sum_out overlap")
    _check_cuda(x, weight, residual, *outs)


def rms_norm_nhwc(x, weight=None, *, eps=1e-6, residual=None, out=None, sum_out=None, return_rstd=False, stream=None):
    """Root-mean-square norm of the pixels (rows of C channels) of
    channels-last X[.., C], of X + residual where a residual is given: float32,
    float16 or bfloat16, weight [C] in X's dtype or float32.  Tensors that are
    not contiguous are copied first.  ``out`` and ``sum_out`` may each be X or
    the residual, but not overlap one another.

    Returns Y; with a residual (Y, sum), sum being X + residual rounded (Y comes
    from the unrounded sum); with ``return_rstd`` also rstd, float32 [..],
    which rms_norm_nhwc_backward takes."""
    r = _rms_of(x, weight, 0, eps)
    if sum_out is not None and residual is None:
        raise ValueError("sum_out needs a residual")
    _rms_inputs(x, weight, residual, out, sum_out)

    def call(raw):
        xc = x.contiguous()
        w = None if weight is None else weight.contiguous()
        h = s = None
        if residual is not None:
            h = residual.contiguous()
            s = torch.empty_like(xc) if sum_out is None else sum_out
        y = torch.empty_like(xc) if out is None else out
        rstd = xc.new_empty(r.rows_shape, dtype=torch.float32) if return_rstd else None
        st = lib().ct_rms_norm(r.desc, xc.data_ptr(), _addr(h), _addr(w), y.data_ptr(), _addr(s), _addr(rstd), raw)
        if st != CT_OK:
            raise CtError(st, "ct_rms_norm")
        if out is not None or sum_out is not None:
            _written(out, sum_out)
        if residual is None:
            return (y, rstd) if return_rstd else y
        return (y, s, rstd) if return_rstd else (y, s)

    return _run_on(call, x, stream)


def rms_norm_nhwc_e4m3(x, weight=None, *, block=None, eps=1e-6, residual=None, sum_out=None, return_rstd=False,
                       stream=None):
    """rms_norm_nhwc with its output in 8 bits for a matrix product that takes
    them: q (float8_e4m3fn, X's shape) and scale (float32), q * scale being the
    value.  A scale serves a pixel (scale [..]) or ``block`` of its channels,
    32, 64 or 128 (scale [.., ceil(C / block)]), and is the largest magnitude
    there / 448.  A block with a NaN or an infinity in it has a NaN scale.

    Returns (q, scale), then sum where there is a residual and rstd with
    ``return_rstd``, as rms_norm_nhwc does."""
    r = _rms_of(x, weight, 0 if block is None else block, eps)
    if sum_out is not None and residual is None:
        raise ValueError("sum_out needs a residual")
    _rms_inputs(x, weight, residual, sum_out)

    def call(raw):
        xc = x.contiguous()
        w = None if weight is None else weight.contiguous()
        h = s = None
        if residual is not None:
            h = residual.contiguous()
            s = torch.empty_like(xc) if sum_out is None else sum_out
        q = xc.new_empty(xc.shape, dtype=torch.float8_e4m3fn)
        scale = xc.new_empty(r.scale_shape, dtype=torch.float32)
        rstd = xc.new_empty(r.rows_shape, dtype=torch.float32) if return_rstd else None
        st = lib().ct_rms_norm_e4m3(r.desc, xc.data_ptr(), _addr(h), _addr(w), q.data_ptr(), scale.data_ptr(),
                                    _addr(s), _addr(rstd), raw)
        if st != CT_OK:
            raise CtError(st, "ct_rms_norm_e4m3")
        if sum_out is not None:
            _written(sum_out)
        out = (q, scale) if residual is None else (q, scale, s)
        return out + (rstd,) if return_rstd else out

    return _run_on(call, x, stream)


def rms_norm_nhwc_backward(dy, x, rstd, weight=None, *, dsum=None, need_x_grad=True, stream=None):
    """Gradients (dx, dweight) of rms_norm_nhwc at dy.  X is what was normed
    (the returned sum where there was a residual), rstd as the forward call
    gave it.  dx is the gradient in X and in the residual alike; ``dsum``, the
    gradient that reaches the sum on its own way, is added to it.  None for dx
    without ``need_x_grad``, and for the gradient of a weight that is None."""
    r = _rms_of(x, weight, 0, 0.0)
    check_like(dy, "dy", x)
    if dsum is not None:
        check_like(dsum, "dsum", x)
    if rstd.dtype != torch.float32 or rstd.shape != r.rows_shape or rstd.device != x.device:
        raise ValueError("rstd must be a float32 tensor of shape %s on %s" % (list(r.rows_shape), x.device))
    _check_cuda(x, dy, rstd, weight, dsum)

    def call(raw):
        xc, dyc, rs = x.contiguous(), dy.contiguous(), rstd.contiguous()
        w = None if weight is None else weight.contiguous()
        d = None if dsum is None else dsum.contiguous()
        dx = torch.empty_like(xc) if need_x_grad else None
        dweight = ws = None
        if w is not None:
            dweight = torch.empty_like(w)
            ws = xc.new_empty((r.backward_bytes,), dtype=torch.uint8)
        st = lib().ct_rms_norm_backward(r.desc, dyc.data_ptr(), xc.data_ptr(), rs.data_ptr(), _addr(w), _addr(d),
                                        _addr(dx), _addr(dweight), _addr(ws), raw)
        if st != CT_OK:
            raise CtError(st, "ct_rms_norm_backward")
        return dx, dweight

    return _run_on(call, x, stream)


# ---- rotary positions ---------------------------------------------------------

PAIRS = {"adjacent": 0, "halves": 1}
POSITION_DTYPE = {torch.int32: 1, torch.int64: 2, torch.float32: 3}


def _head_strides(shape, stride):
    """(image, pixel, head) strides of [N, D1.., heads, dim], or None where the
    pixels are not one stride apart or a head's elements are not neighbours."""
    if shape[-1] > 1 and stride[-1] != 1:
        return None
    pixel = span = None
    for size, step in zip(reversed(shape[1:-2]), reversed(stride[1:-2])):
        if size == 1:
            continue
        if pixel is None:
            pixel = span = step
        elif step != span:
            return None
        span *= size
    return stride[0], 0 if pixel is None else pixel, stride[-2]


def _extent(t):
    """First byte of a tensor and the one behind its last (no negative strides)."""
    a = t.data_ptr()
    return a, a + (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size()


def check_rotary(x, sections, base, pairs, positions):
    """Refuse arguments that the rotation cannot take."""
    if x.dtype not in NORM_DTYPE:
        raise ValueError("X must be float32, float16 or bfloat16, not %s" % x.dtype)
    if not 1 <= len(sections) <= 3:
        raise ValueError("sections must name 1 to 3 axes, not %d" % len(sections))
    if x.dim() < 4:
        raise ValueError("X must be [N, D.., heads, dim], it has shape %s" % list(x.shape))
    for v in sections:
        if v != int(v) or v < 0 or v % 2 != 0:
            raise ValueError("each section must be an even number of elements, not %r" % (v,))
    if sum(sections) > min(x.shape[-1], 512):
        raise ValueError("sections of %d elements do not fit a head of %d (and 512)" % (sum(sections), x.shape[-1]))
    if pairs not in PAIRS:
        raise ValueError("pairs must be one of %s, not %r" % (sorted(PAIRS), pairs))
    if not 0.0 < base < math.inf:
        raise ValueError("base must be positive and finite, not %r" % (base,))
    if positions is None:
        if x.dim() != 3 + len(sections):
            raise ValueError("X of shape %s does not have the %d pixel axes of sections; give positions"
                             % (list(x.shape), len(sections)))
        return
    if positions.dtype not in POSITION_DTYPE:
        raise ValueError("positions must be int32, int64 or float32, not %s" % positions.dtype)
    want = tuple(x.shape[1:-2]) + (len(sections),)
    if positions.device != x.device or tuple(positions.shape) not in (want, (x.shape[0],) + want):
        raise ValueError("positions must have shape %s or %s on %s"
                         % (list(want), [x.shape[0]] + list(want), x.device))


class _Rotary:
    """A rotation's descriptor, for one set of sizes, types and strides."""

    def __init__(self, x, out, sections, base, pairs, positions, inverse):
        check_rotary(x, sections, base, pairs, positions)
        xs = _head_strides(x.shape, x.stride())
        self.copy = xs is None          # X is copied first, to dense heads
        dense = torch.empty(x.shape, device="meta").stride()
        if xs is None:
            xs = _head_strides(x.shape, dense)
        ys = _head_strides(x.shape, dense if out is None else out.stride())
        if ys is None:
            raise ValueError("out's pixels must be one stride apart, and a head's elements neighbours")
        d = self.desc = ct_rotary_desc(NORM_DTYPE[x.dtype], len(sections), PAIRS[pairs], inverse)
        d.N, d.heads, d.dim, d.base = x.shape[0], x.shape[-2], x.shape[-1], float(base)
        grid = list(x.shape[1:-2])
        if positions is not None:
            d.position_type = POSITION_DTYPE[positions.dtype]
            d.position_images = int(positions.dim() == x.dim() - 1)
            grid = [math.prod(grid)] + [1] * (len(sections) - 1)
        for a, v in enumerate(sections):
            d.grid[a], d.sections[a] = grid[a], int(v)
        for a in range(3):
            d.x_strides[a], d.y_strides[a] = xs[a], ys[a]


_ROTARY = {}


def _rotate(x, sections, base, pairs, positions, out, stream, inverse):
    if out is not None:
        check_like(out, "out", x)
    key = (x.shape, x.stride(), x.dtype, tuple(sections), base, pairs, inverse,
           None if out is None else out.stride(), None if positions is None else (positions.shape, positions.dtype))
    try:
        r = _ROTARY[key]
    except (KeyError, TypeError):
        r = _Rotary(x, out, sections, base, pairs, positions, inverse)
        if _kept_by_value(base, *sections):
            if len(_ROTARY) >= 1024:
                _ROTARY.clear()
            _ROTARY[key] = r
    if positions is not None and positions.device != x.device:
        check_rotary(x, sections, base, pairs, positions)
    if out is not None:
        o0, o1 = _extent(out)
        for t in (x, positions):
            if t is None or t.numel() == 0:
                continue
            t0, t1 = _extent(t)
            if t0 < o1 and o0 < t1 and not (t is x and t0 == o0 and x.stride() == out.stride()):
                raise ValueError("out overlaps an input")
    _check_cuda(x, positions, out)

    def call(raw):
        xc = x.contiguous() if r.copy else x
        pos = None if positions is None else positions.contiguous()
        if out is not None:
            y = out
        elif xc.is_contiguous():
            y = torch.empty_like(xc)
        else:
            y = torch.empty(xc.shape, dtype=xc.dtype, device=xc.device)
        st = lib().ct_rotary(r.desc, xc.data_ptr(), _addr(pos), y.data_ptr(), raw)
        if st != CT_OK:
            raise CtError(st, "ct_rotary")
        if out is not None:
            _written(out)
        return y

    return _run_on(call, x, stream)


def rotary_nhwc(x, sections, *, base=10000.0, pairs="adjacent", positions=None, out=None, stream=None):
    """Rotary positions of heads X[N, D1.., heads, dim] on 1 to 3 axes: the first
    sum(sections) elements of each head are rotated in pairs, sections[a] of
    them (even) by the position on axis a; the rest stay as they are.  float32,
    float16 or bfloat16.  Pair i is elements 2i and 2i + 1 ("adjacent") or i
    and i + sum(sections) / 2 ("halves"); the first pairs are axis 0's, and the
    j-th pair of axis a turns by position * base^(-2j / sections[a]).

    Positions are the pixels' indices, or ``positions`` (int32, int64 or
    float32), [D1.., axes] for all images or [N, D1.., axes].  X may be a slice
    (the queries and keys of a packed projection) or have its heads outside its
    pixels in memory, without a copy, where its pixels are one stride apart;
    other layouts are copied.  ``out`` may be X."""
    return _rotate(x, sections, base, pairs, positions, out, stream, 0)


def rotary_nhwc_backward(dy, sections, *, base=10000.0, pairs="adjacent", positions=None, out=None, stream=None):
    """The gradient of rotary_nhwc in X at dy (dy rotated back), for the
    sections, base, pairs and positions of the forward call."""
    return _rotate(dy, sections, base, pairs, positions, out, stream, 1)


# ---- a training step's end: the gradients' norm, AdamW ---------------------------

BLOCK = 256     # elements of a block of AdamW's states


# What a step asks of each of its tensors, as functions that map() runs over a
# list: a step of dozens of small tensors is bound by these questions.
_shape, _dtype = torch.Tensor.shape.__get__, torch.Tensor.dtype.__get__
_numel, _device, _dense, _where = (torch.Tensor.numel, torch.Tensor.get_device, torch.Tensor.is_contiguous,
                                   torch.Tensor.data_ptr)


def _pointers(addresses):
    """A host array of device addresses (keep it while its address is used)."""
    return array.array("Q", addresses)


def _check_grad(g, name):
    if not g.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if g.dtype not in NORM_DTYPE:
        raise ValueError("%s must be float32, float16 or bfloat16, not %s" % (name, g.dtype))
    if g.layout != torch.strided:
        raise ValueError("%s must be a dense tensor" % name)


def _check_derivatives(grads):
    """Gradients that carry derivatives of their own are refused, as inputs of the other calls are (_check_cuda)."""
    if forward_ad._current_level >= 0:
        for g in grads:
            if forward_ad.unpack_dual(g).tangent is not None:
                raise ValueError("a gradient carries a forward-mode tangent, and this call computes none")
    if torch.is_grad_enabled() and torch._C._any_requires_grad(*grads):
        raise ValueError("a gradient requires a gradient itself, and this call records none: call it under "
                         "torch.no_grad(), or detach it")


_GRADS = {}


def _grads_of(grads):
    """The descriptors of gradients that lie on one device, and the workspace's
    size (made once per sizes and types)."""
    key = (tuple(map(_numel, grads)), tuple(map(_dtype, grads)), tuple(map(_device, grads)))
    try:
        return _GRADS[key]
    except KeyError:
        pass
    for i, g in enumerate(grads):
        _check_grad(g, "gradient %d" % i)
        if g.device != grads[0].device:
            raise ValueError("gradient %d is on %s, the first on %s" % (i, g.device, grads[0].device))
    shapes = (ct_param * len(grads))(*[ct_param(g.numel(), NORM_DTYPE[g.dtype], NORM_DTYPE[g.dtype], 0.0)
                                       for g in grads])
    n = ctypes.c_size_t()
    st = lib().ct_grad_norm_workspace_bytes(len(grads), ctypes.byref(n))
    if st != CT_OK:
        raise CtError(st, "ct_grad_norm_workspace_bytes")
    if len(_GRADS) >= 64:
        _GRADS.clear()
    _GRADS[key] = shapes, n.value
    return _GRADS[key]


def grad_norm(grads, max_norm=None, *, stream=None):
    """The 2-norm of all gradients together (float32, float16 and bfloat16 may
    be mixed; None entries count nothing) and the scale that clips it to
    max_norm, float32 tensors without dimensions on the gradients' device:
    scale = min(1, max_norm / norm), 0 where the norm is not finite.  Give the
    scale to AdamW.step: nothing waits for it, and 0 skips the step."""
    grads = [g for g in grads if g is not None]
    if not grads:
        raise ValueError("there is no gradient")
    if max_norm is None:
        max_norm = math.inf
    if not max_norm > 0.0:
        raise ValueError("max_norm must be positive, not %r" % (max_norm,))
    _check_derivatives(grads)
    shapes, bytes_ = _grads_of(grads)

    def call(raw):
        dense = grads if all(map(_dense, grads)) else [g.contiguous() for g in grads]
        at = _pointers(map(_where, dense))
        dev = grads[0].device
        out = torch.empty(2, dtype=torch.float32, device=dev)
        ws = torch.empty(bytes_, dtype=torch.uint8, device=dev)
        st = lib().ct_grad_norm(len(dense), shapes, at.buffer_info()[0], max_norm, out.data_ptr(),
                                out.data_ptr() + 4, ws.data_ptr(), raw)
        if st != CT_OK:
            raise CtError(st, "ct_grad_norm")
        return out.unbind()

    return _run_on(call, grads[0], stream)


class AdamW:
    """AdamW over many tensors, one launch for up to 512 of them.

    ``params`` are contiguous CUDA tensors (float32, float16, bfloat16; mixed)
    on one device, updated in place; ``weight_decay`` is a number or one for each.
    Parameters of 16 bits get float32 masters, which the updates work on.
    ``bits=8`` holds the states in 8 bits, rounded at random by ``seed``.

    The states are tensors of this object, to be saved and copied back for a
    restart together with ``steps``: exp_avg and exp_avg_sq, all parameters one
    after the other, each from a multiple of 256 elements on (float32, or with
    bits=8 float8_e4m3fn codes of exp_avg and of the square root of exp_avg_sq,
    under exp_avg_scale and exp_avg_sq_scale, a scale for 256), and master
    (None without parameters of 16 bits).  ``lr`` may be changed between steps,
    and be a float32 CUDA tensor of one element, which is read on the device."""

    def __init__(self, params, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, seed=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("there is no parameter")
        if bits not in (32, 8):
            raise ValueError("bits must be 32 or 8, not %r" % (bits,))
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be in [0, 2^64)")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError("betas must be in [0, 1), not %r" % (betas,))
        if not 2.0 ** -126 <= eps < math.inf:
            raise ValueError("eps must be positive and finite, not %r" % (eps,))
        n = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(decay) != n or not all(0.0 <= v < math.inf for v in decay):
            raise ValueError("weight_decay must be a number >= 0, or one for each of %d parameters" % n)
        for i, p in enumerate(self.params):
            _check_grad(p, "parameter %d" % i)
            if p.device != self.params[0].device:
                raise ValueError("parameter %d is on %s, the first on %s" % (i, p.device, self.params[0].device))
        self.device = self.params[0].device
        self.lr, self.betas, self.eps, self.bits, self.seed, self.steps = lr, tuple(betas), eps, int(bits), seed, 0
        self._sizes = [p.numel() for p in self.params]
        self._dtypes = [p.dtype for p in self.params]
        self._shapes = [p.shape for p in self.params]
        self._at = self._places()
        self._decay = decay
        self._meta = self._table = None
        self._desc = ct_adamw_desc(int(bits))
        blocks = [-(-k // BLOCK) for k in self._sizes]
        total = sum(blocks)
        kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
        self.exp_avg = torch.zeros(total * BLOCK, dtype=torch.float32 if bits == 32 else torch.uint8,
                                   device=self.device).view(kind)
        self.exp_avg_sq = torch.zeros_like(self.exp_avg.view(torch.uint8)).view(kind)
        self.exp_avg_scale = self.exp_avg_sq_scale = self.master = None
        if bits == 8:
            self.exp_avg_scale = torch.zeros(total, dtype=torch.float32, device=self.device)
            self.exp_avg_sq_scale = torch.zeros_like(self.exp_avg_scale)
        low = [i for i, p in enumerate(self.params) if p.dtype != torch.float32]
        if low:
            self.master = torch.zeros(sum(blocks[i] for i in low) * BLOCK, dtype=torch.float32, device=self.device)
            at = 0
            for i in low:
                self.master[at:at + self._sizes[i]].copy_(self.params[i].detach().reshape(-1))
                at += blocks[i] * BLOCK
        self._kept = [t.numel() if t is not None else 0 for t in self._states()]
        self._kept_at = self._kept_places()
        self._kept_as = self._kept_looks()

    def _states(self):
        return self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale, self.master

    def _kept_looks(self):
        """What tells whether the states still are those that _kept_places saw."""
        return [None if t is None else (t.data_ptr(), t.numel(), t.dtype, t.is_contiguous()) for t in self._states()]

    def _kept_places(self):
        """The states' addresses; a tensor in the place of one has to be like it."""
        kind = torch.float32 if self.bits == 32 else torch.float8_e4m3fn
        for t, n, name, dtype in zip(self._states(), self._kept,
                                     ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master"),
                                     (kind, kind) + 3 * (torch.float32,)):
            if (0 if t is None else t.numel()) != n or t is not None and (
                    t.dtype != dtype or t.device != self.device or not t.is_contiguous()):
                raise ValueError("%s must be a contiguous %s tensor of %d elements on %s" % (name, dtype, n, self.device))
        return [_addr(t) for t in self._states()]

    def _places(self):
        """The parameters' addresses, as bytes; they have to be dense and apart."""
        for i, p in enumerate(self.params):
            if not p.is_contiguous():
                raise ValueError("parameter %d must be contiguous" % i)
            if p.shape != self._shapes[i] or p.dtype != self._dtypes[i] or p.device != self.device:
                raise ValueError("parameter %d has another shape, type or device than it had" % i)
        spans = sorted(_extent(p) for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("two parameters overlap")
        return _pointers(map(_where, self.params)).tobytes()

    def _grads(self, grads):
        """Check the gradients and make their descriptors; None entries stay."""
        kinds = []
        for i, (g, shape, dtype) in enumerate(zip(grads, self._shapes, self._dtypes)):
            if g is None:
                kinds.append(dtype)
                continue
            _check_grad(g, "gradient %d" % i)
            if g.shape != shape or g.device != self.device or g.dtype not in (dtype, torch.float32):
                raise ValueError("gradient %d must be a %s or float32 tensor of shape %s on %s"
                                 % (i, dtype, list(shape), self.device))
            kinds.append(g.dtype)
        self._table = (ct_param * len(kinds))(*[
            ct_param(n, NORM_DTYPE[d], NORM_DTYPE[k], w)
            for n, d, k, w in zip(self._sizes, self._dtypes, kinds, self._decay)])

    def _scalar(self, t, name, dtype):
        if t.dtype != dtype or t.numel() != 1 or t.device != self.device:
            raise ValueError("%s must be a %s tensor of one element on %s" % (name, dtype, self.device))
        return t.data_ptr()

    def step(self, grads, *, grad_scale=None, step=None, stream=None):
        """One update by ``grads``, a gradient for each parameter in its dtype
        or float32 (None leaves a parameter and its states as they are).

        ``grad_scale``, a float32 CUDA tensor of one element (grad_norm's),
        multiplies the gradients; one that is not positive and finite skips the
        update.  ``steps`` counts the updates, skipped ones too; ``step``, an
        int64 CUDA tensor of one element, is the number of this update (1 for
        the first) in its place, read on the device: a captured graph needs it,
        and counts with it.  A step below 1, and an lr on the device that is
        negative or not finite, skip the update too.  Gradients may not overlap
        parameters or states."""
        grads = list(grads)
        params = self.params
        if len(params) != len(self._sizes):
            raise ValueError("%d parameters, not the %d that the states are for" % (len(params), len(self._sizes)))
        if len(grads) != len(params):
            raise ValueError("%d gradients for %d parameters" % (len(grads), len(params)))
        try:
            meta = [list(map(_shape, grads)), list(map(_dtype, grads)), list(map(_device, grads))]
        except TypeError:       # None entries
            meta = None
        if meta is None or meta != self._meta:
            self._meta = None
            self._grads(grads)
            self._meta = meta
        _check_derivatives(grads if meta is not None else [g for g in grads if g is not None])
        # all that the kernel relies on: a parameter can become another at its old address
        to = _pointers(map(_where, params))
        if (to.tobytes() != self._at or list(map(_numel, params)) != self._sizes
                or list(map(_dtype, params)) != self._dtypes or False in map(_dense, params)):
            self._at = self._places()
        if self._kept_looks() != self._kept_as:
            self._kept_at = self._kept_places()
            self._kept_as = self._kept_looks()
        d, lr = self._desc, self.lr
        d.beta1, d.beta2 = self.betas
        d.eps, d.seed = self.eps, self.seed
        d.grad_scale = None if grad_scale is None else self._scalar(grad_scale, "grad_scale", torch.float32)
        d.step_device = None if step is None else self._scalar(step, "step", torch.int64)
        if isinstance(lr, torch.Tensor):
            d.lr_device, d.lr = self._scalar(lr, "lr", torch.float32), 0.0
        else:
            if not 0.0 <= lr < math.inf:
                raise ValueError("lr must be >= 0 and finite, not %r" % (lr,))
            d.lr_device, d.lr = None, lr
        d.step = self.steps + 1

        def call(raw):
            if step is None and torch.cuda.is_current_stream_capturing():
                raise ValueError("a captured step would keep its number: give step, a CUDA tensor")
            if meta is None:
                dense = [None if g is None else g.contiguous() for g in grads]
                at = _pointers([0 if g is None else g.data_ptr() for g in dense])
            else:
                dense = grads if all(map(_dense, grads)) else [g.contiguous() for g in grads]
                at = _pointers(map(_where, dense))
            st = lib().ct_adamw(d, len(dense), self._table, to.buffer_info()[0], at.buffer_info()[0],
                                *self._kept_at, raw)
            if st != CT_OK:
                raise CtError(st, "ct_adamw")

        _run_on(call, self.exp_avg, stream)
        if step is None:
            self.steps += 1
        # those that stay as they are stay valid for what saved them
        torch.autograd.graph.increment_version(
            params if meta is not None else [p for p, g in zip(params, grads) if g is not None])
