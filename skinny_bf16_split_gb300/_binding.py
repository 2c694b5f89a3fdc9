"""ctypes binding of the C ABI in include/dep_projection.h (marshalling only).

Every function keeps the C name and takes the same arguments; tensors may be
passed as torch tensors (BF16, contiguous, on the plan's device) or as raw
integer addresses.  Each step of the projection runs in the library's CUDA
kernels; nothing here computes.  The library must have been built (see
``skinny_bf16_split_gb300.build``): there is no fallback, and loading fails
loudly when it is missing.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdep_projection.so")

DEP_OK = 0
DEP_ERR_INVALID_ARG = 1
DEP_ERR_UNSUPPORTED = 2
DEP_ERR_MISALIGNED = 3
DEP_ERR_CUDA = 4
DEP_ERR_OOM = 5
DEP_ERR_TIMEOUT = 6
DEP_ERR_INTERNAL = 7
DEP_ERR_IO = 8

DEP_KIND_SPLITK_FMA = 1
DEP_KIND_TC = 2
DEP_KIND_ROWS = 3
DEP_KIND_TC_SPLIT = 4
DEP_KIND_TC_WIDE = 5
DEP_KIND_TC_CLUSTER = 6
DEP_KIND_TC_XM = 7
DEP_KIND_WARP_MMA = 8
DEP_PLAN_DEFAULT = 0
DEP_PLAN_TUNE = 1
DEP_PLAN_PDL = 2
DEP_PLAN_KEEP_PIECES = 4

DEP_QUANT_NONE = 0
DEP_QUANT_INT8 = 1
DEP_QUANT_E4M3 = 2
DEP_QUANT_GROUP = 128
DEP_NORM_MAX_COLS = 65536
DEP_DELTA_CHANNEL = 1
DEP_DELTA_L2NORM = 2

DEP_DEV_TIMEOUT_PRODUCER = 1
DEP_DEV_TIMEOUT_CONSUMER = 2
DEP_DEV_TIMEOUT_MMA = 3
DEP_DEV_TIMEOUT_EPILOGUE = 4
DEP_DEV_BOUNDS = 5

# Every symbol include/dep_projection.h declares.
EXPORTS = (
    "dep_projection_plan", "dep_projection_plan_host", "dep_projection_run",
    "dep_projection_run_tactic", "dep_projection_run_host", "dep_projection_plan_query",
    "dep_projection_plan_table", "dep_projection_plan_set", "dep_projection_plan_workspace",
    "dep_projection_plan_save", "dep_projection_plan_load", "dep_projection_plan_destroy",
    "dep_projection_device_status", "dep_projection_selftest_timeout", "dep_bins_index",
    "dep_status_string", "dep_projection_version", "dep_projection_run_static",
    "dep_projection_plan_partials", "dep_projection_plan_exchange", "dep_projection_probe_read",
    "dep_projection_plan_selftest_exchange",
    "dep_add_rms_norm", "dep_quantize_rows", "dep_delta_rule", "dep_delta_workspace", "dep_int8_plan", "dep_int8_run",
    "dep_int8_plan_workspace", "dep_int8_device_status", "dep_int8_plan_destroy",
)


class dep_tactic_t(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in
                ("max_rows", "kind", "ctas", "tile_n", "tile_k", "stages", "cols", "splits")]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}

    def __repr__(self):
        return f"dep_tactic_t({self.as_dict()})"


class dep_norm_args_t(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_void_p) for name in ("x", "residual", "weight", "residual_out", "out", "scale")]
                + [(name, ctypes.c_int64) for name in
                   ("x_stride", "residual_stride", "residual_out_stride", "out_stride", "rows", "cols")]
                + [("quant", ctypes.c_int32), ("eps", ctypes.c_float)])


class dep_delta_args_t(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_void_p) for name in
                 ("q", "k", "v", "g", "beta", "state_in", "state_out", "o", "cu_seqlens", "slots")]
                + [(name, ctypes.c_int64) for name in
                   ("q_stride", "k_stride", "v_stride", "g_stride", "beta_stride", "o_stride", "tokens", "n_states")]
                + [(name, ctypes.c_int32) for name in ("n_seq", "Hq", "Hv", "Dk", "Dv")]
                + [("flags", ctypes.c_uint32), ("scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
                   ("workspace_bytes", ctypes.c_int64)])


class DepError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dep_status_string(status)} (status {status})")


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with skinny_bf16_split_gb300.build.build() "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
    P = ctypes.POINTER
    sig = {
        "dep_projection_plan": ([i64, i64, P(i32), i32, u32, P(vp)], i32),
        "dep_projection_plan_host": ([i64, i64, P(i32), i32, i32, P(vp)], i32),
        "dep_projection_run": ([vp, vp, vp, vp, i32, vp], i32),
        "dep_projection_run_tactic": ([vp, P(dep_tactic_t), vp, vp, vp, i32, vp], i32),
        "dep_projection_run_host": ([vp, vp, vp, vp, i32, vp], i32),
        "dep_projection_plan_query": ([vp, i32, P(dep_tactic_t)], i32),
        "dep_projection_plan_table": ([vp, P(dep_tactic_t), i32, P(i32)], i32),
        "dep_projection_plan_set": ([vp, P(dep_tactic_t)], i32),
        "dep_projection_plan_workspace": ([vp, P(ctypes.c_size_t)], i32),
        "dep_projection_plan_save": ([vp, ctypes.c_char_p], i32),
        "dep_projection_plan_load": ([ctypes.c_char_p, i64, i64, P(vp)], i32),
        "dep_projection_plan_destroy": ([vp], None),
        "dep_projection_device_status": ([vp, vp, P(i32)], i32),
        "dep_projection_selftest_timeout": ([i32, P(i32)], i32),
        "dep_bins_index": ([P(i32), i32, i32], i32),
        "dep_status_string": ([i32], ctypes.c_char_p),
        "dep_projection_version": ([], i32),
        "dep_projection_run_static": ([vp, vp, vp, i64, i64, i32, vp], i32),
        "dep_projection_plan_partials": ([vp, vp, ctypes.c_size_t, P(ctypes.c_size_t)], i32),
        "dep_projection_plan_exchange": ([vp, vp, ctypes.c_size_t, P(ctypes.c_size_t)], i32),
        "dep_projection_probe_read": ([vp, ctypes.c_size_t, vp, vp], i32),
        "dep_projection_plan_selftest_exchange": ([vp, i32, vp], i32),
        "dep_add_rms_norm": ([P(dep_norm_args_t), vp], i32),
        "dep_quantize_rows": ([P(dep_norm_args_t), vp], i32),
        "dep_delta_rule": ([P(dep_delta_args_t), vp], i32),
        "dep_delta_workspace": ([P(dep_delta_args_t), P(ctypes.c_int64)], i32),
        "dep_int8_plan": ([i64, i64, i32, P(vp)], i32),
        "dep_int8_run": ([vp, vp, vp, vp, vp, vp, i32, vp], i32),
        "dep_int8_plan_workspace": ([vp, P(ctypes.c_size_t)], i32),
        "dep_int8_device_status": ([vp, vp, P(i32)], i32),
        "dep_int8_plan_destroy": ([vp], None),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(status: int, where: str):
    if status != DEP_OK:
        raise DepError(status, where)


def _ptr(t):
    """Device address of a tensor (or an int address as is)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _i32_array(values):
    values = list(values)
    return (ctypes.c_int32 * max(1, len(values)))(*values), len(values)


# ---- the C functions, same names -------------------------------------------

def dep_status_string(status: int) -> str:
    return lib().dep_status_string(status).decode()


def dep_projection_version() -> int:
    return lib().dep_projection_version()


def dep_bins_index(keys, B: int) -> int:
    arr, n = _i32_array(keys)
    return lib().dep_bins_index(arr, n, B)


def dep_projection_plan(N: int, K: int, batches=(), flags: int = DEP_PLAN_DEFAULT):
    arr, n = _i32_array(batches)
    out = ctypes.c_void_p()
    _check(lib().dep_projection_plan(N, K, arr, n, flags, ctypes.byref(out)), "dep_projection_plan")
    return out.value


def dep_projection_plan_host(N: int, K: int, batches=(), sm_count: int = 152):
    arr, n = _i32_array(batches)
    out = ctypes.c_void_p()
    _check(lib().dep_projection_plan_host(N, K, arr, n, sm_count, ctypes.byref(out)),
           "dep_projection_plan_host")
    return out.value


def dep_projection_run(plan, x, W, y, B: int | None = None, stream=None) -> None:
    if B is None:
        B = x.shape[0]
    _check(lib().dep_projection_run(plan, _ptr(x), _ptr(W), _ptr(y), B, _stream(stream)),
           "dep_projection_run")


def dep_projection_run_tactic(plan, tactic: dep_tactic_t, x, W, y, B: int | None = None,
                              stream=None) -> None:
    if B is None:
        B = x.shape[0]
    _check(lib().dep_projection_run_tactic(plan, ctypes.byref(tactic), _ptr(x), _ptr(W), _ptr(y),
                                           B, _stream(stream)), "dep_projection_run_tactic")


def dep_projection_run_host(plan, x_host, W, y_host, B: int | None = None, stream=None) -> None:
    if B is None:
        B = x_host.shape[0]
    _check(lib().dep_projection_run_host(plan, _ptr(x_host), _ptr(W), _ptr(y_host), B,
                                         _stream(stream)), "dep_projection_run_host")


def dep_projection_plan_query(plan, B: int) -> dep_tactic_t:
    t = dep_tactic_t()
    _check(lib().dep_projection_plan_query(plan, B, ctypes.byref(t)), "dep_projection_plan_query")
    return t


def dep_projection_plan_table(plan) -> list:
    n = ctypes.c_int32()
    _check(lib().dep_projection_plan_table(plan, None, 0, ctypes.byref(n)), "dep_projection_plan_table")
    arr = (dep_tactic_t * max(1, n.value))()
    _check(lib().dep_projection_plan_table(plan, arr, n.value, ctypes.byref(n)),
           "dep_projection_plan_table")
    return [arr[i] for i in range(n.value)]


def dep_projection_plan_set(plan, tactic: dep_tactic_t) -> None:
    _check(lib().dep_projection_plan_set(plan, ctypes.byref(tactic)), "dep_projection_plan_set")


def dep_projection_plan_workspace(plan) -> int:
    b = ctypes.c_size_t()
    _check(lib().dep_projection_plan_workspace(plan, ctypes.byref(b)), "dep_projection_plan_workspace")
    return b.value


def dep_projection_plan_partials(plan, count: int):
    """The first `count` FP32 split-K partials of the plan's workspace (numpy)."""
    import numpy as np
    out = np.empty(count, dtype=np.float32)
    n = ctypes.c_size_t()
    _check(lib().dep_projection_plan_partials(plan, out.ctypes.data, out.nbytes, ctypes.byref(n)),
           "dep_projection_plan_partials")
    return out[: n.value // 4]


def dep_projection_plan_exchange(plan, count: int):
    """The first `count` 64-bit K-piece exchange words of the plan (numpy uint64)."""
    import numpy as np
    out = np.empty(count, dtype=np.uint64)
    n = ctypes.c_size_t()
    _check(lib().dep_projection_plan_exchange(plan, out.ctypes.data, out.nbytes, ctypes.byref(n)),
           "dep_projection_plan_exchange")
    return out[: n.value // 8]


def dep_projection_plan_save(plan, path: str) -> None:
    _check(lib().dep_projection_plan_save(plan, os.fsencode(path)), "dep_projection_plan_save")


def dep_projection_plan_load(path: str, N: int, K: int):
    out = ctypes.c_void_p()
    _check(lib().dep_projection_plan_load(os.fsencode(path), N, K, ctypes.byref(out)),
           "dep_projection_plan_load")
    return out.value


def dep_projection_plan_destroy(plan) -> None:
    lib().dep_projection_plan_destroy(plan)


def dep_projection_device_status(plan, stream=None) -> int:
    code = ctypes.c_int32()
    st = lib().dep_projection_device_status(plan, _stream(stream), ctypes.byref(code))
    if st not in (DEP_OK, DEP_ERR_TIMEOUT):
        _check(st, "dep_projection_device_status")
    return code.value


def dep_projection_selftest_timeout(limit_us: int) -> int:
    code = ctypes.c_int32()
    _check(lib().dep_projection_selftest_timeout(limit_us, ctypes.byref(code)),
           "dep_projection_selftest_timeout")
    return code.value


def dep_projection_run_static(x, W, y, N: int | None = None, K: int | None = None,
                              B: int | None = None, stream=None) -> None:
    """The no-allocation entry point (see include/dep_projection.h): for callers
    that must not allocate device memory, so cannot hold a plan."""
    if N is None:
        N, K = W.shape
    if B is None:
        B = x.shape[0]
    _check(lib().dep_projection_run_static(_ptr(x), _ptr(W), _ptr(y), N, K, B, _stream(stream)),
           "dep_projection_run_static")


def dep_projection_plan_selftest_exchange(plan, limit_us: int, stream=None) -> None:
    """Enqueue the split-K exchange's give-up self-test on the plan's workspace."""
    _check(lib().dep_projection_plan_selftest_exchange(plan, limit_us, _stream(stream)),
           "dep_projection_plan_selftest_exchange")


def dep_projection_probe_read(p, nbytes: int, sink, stream=None) -> None:
    """Read-only streaming pass over nbytes of device memory at p (measurement aid)."""
    _check(lib().dep_projection_probe_read(_ptr(p), nbytes, _ptr(sink), _stream(stream)),
           "dep_projection_probe_read")


def dep_add_rms_norm(args: dep_norm_args_t, stream=None) -> None:
    _check(lib().dep_add_rms_norm(ctypes.byref(args), _stream(stream)), "dep_add_rms_norm")


def dep_quantize_rows(args: dep_norm_args_t, stream=None) -> None:
    _check(lib().dep_quantize_rows(ctypes.byref(args), _stream(stream)), "dep_quantize_rows")


def dep_delta_rule(args: dep_delta_args_t, stream=None) -> None:
    _check(lib().dep_delta_rule(ctypes.byref(args), _stream(stream)), "dep_delta_rule")


def dep_int8_plan(N: int, K: int, max_rows: int = 256):
    out = ctypes.c_void_p()
    _check(lib().dep_int8_plan(N, K, max_rows, ctypes.byref(out)), "dep_int8_plan")
    return out.value


def dep_int8_run(plan, x, x_scale, W, w_scale, y, B: int | None = None, stream=None) -> None:
    if B is None:
        B = x.shape[0]
    _check(lib().dep_int8_run(plan, _ptr(x), _ptr(x_scale), _ptr(W), _ptr(w_scale), _ptr(y), B, _stream(stream)),
           "dep_int8_run")


def dep_delta_workspace(args: dep_delta_args_t) -> int:
    b = ctypes.c_int64()
    _check(lib().dep_delta_workspace(ctypes.byref(args), ctypes.byref(b)), "dep_delta_workspace")
    return b.value


def dep_int8_plan_workspace(plan) -> int:
    b = ctypes.c_size_t()
    _check(lib().dep_int8_plan_workspace(plan, ctypes.byref(b)), "dep_int8_plan_workspace")
    return b.value


def dep_int8_device_status(plan, stream=None) -> int:
    code = ctypes.c_int32()
    st = lib().dep_int8_device_status(plan, _stream(stream), ctypes.byref(code))
    if st not in (DEP_OK, DEP_ERR_TIMEOUT):
        _check(st, "dep_int8_device_status")
    return code.value


def dep_int8_plan_destroy(plan) -> None:
    lib().dep_int8_plan_destroy(plan)


class Projection:
    """A TP1 decode linear over one resident BF16 weight W[N,K]: the library's
    counterpart of DepProjection (runtime.dep page).  ``run(x, out)`` writes
    BF16(x . W^T) into ``out`` (allocated here when omitted) and returns it."""

    def __init__(self, weight, batches=(), flags: int = DEP_PLAN_DEFAULT):
        import torch
        if weight.dtype != torch.bfloat16 or not weight.is_cuda or not weight.is_contiguous():
            raise ValueError("weight must be a contiguous CUDA bfloat16 tensor [N, K]")
        self.weight = weight
        self.N, self.K = weight.shape
        with torch.cuda.device(weight.device):
            self.plan = dep_projection_plan(self.N, self.K, batches, flags)

    def run(self, x, out=None, stream=None):
        import torch
        if x.dtype != torch.bfloat16 or not x.is_contiguous() or x.device != self.weight.device:
            raise ValueError("x must be a contiguous bfloat16 tensor on the weight's device")
        if out is None:
            out = torch.empty((x.shape[0], self.N), dtype=torch.bfloat16, device=x.device)
        dep_projection_run(self.plan, x, self.weight, out, x.shape[0], stream)
        return out

    def tactic(self, B: int) -> dep_tactic_t:
        return dep_projection_plan_query(self.plan, B)

    def close(self):
        if getattr(self, "plan", None):
            dep_projection_plan_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- around the projections ---------------------------------------------------
#
# Calls of a few microseconds of GPU work each: the checks below build no messages
# and no contexts unless they refuse.

_QUANT = {None: DEP_QUANT_NONE, "int8": DEP_QUANT_INT8, "e4m3": DEP_QUANT_E4M3}


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream of the call that writes it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(index, call, args, stream):
    """call(args, stream) with device `index` current; stream None: its current stream."""
    import torch
    if index == torch._C._cuda_getDevice():  # (torch.cuda.current_device takes twice as long)
        call(args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream)
        return
    with torch.cuda.device(index):
        call(args, stream)


def _rows(t, name, dtype, index, shape):
    """Stride between the rows of a matrix whose rows are contiguous."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        row, col = t.stride()
        if col == 1 or shape[1] <= 1:
            return row if shape[0] > 1 else shape[1]
    raise ValueError(f"{name} must be a {dtype} matrix {tuple(shape)} with contiguous rows on cuda:{index}")


def _norm_call(call, x, weight, residual, residual_out, eps, quant, out, out_scale, stream):
    import torch
    if quant not in _QUANT:
        raise ValueError("quant must be None, 'int8' or 'e4m3'")
    shape, dev, bf16 = x.shape, x.get_device(), torch.bfloat16
    if len(shape) != 2 or dev < 0:
        raise ValueError("x must be a CUDA matrix [rows, cols]")
    rows, cols = shape
    w_ptr = r_ptr = ro_ptr = s_ptr = None
    r_stride = ro_stride = 0
    if weight is not None:
        if weight.dtype is not bf16 or weight.get_device() != dev or weight.shape != (cols,) or (
                not weight.is_contiguous()):
            raise ValueError(f"weight must be a contiguous bfloat16 vector of {cols} on cuda:{dev}")
        w_ptr = weight.data_ptr()
    if residual is not None:
        r_ptr, r_stride = residual.data_ptr(), _rows(residual, "residual", bf16, dev, shape)
        if residual_out is None:
            ro_ptr, ro_stride = r_ptr, r_stride
        else:
            ro_ptr, ro_stride = residual_out.data_ptr(), _rows(residual_out, "residual_out", bf16, dev, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    dtype = bf16 if quant is None else torch.int8 if quant == "int8" else torch.float8_e4m3fn
    if out is None:
        out = _empty((rows, cols), dtype, x.device, stream)
    if quant is not None:
        want = (rows,) if quant == "int8" else (rows, -(-cols // DEP_QUANT_GROUP))
        if out_scale is None:
            out_scale = _empty(want, torch.float32, x.device, stream)
        elif out_scale.dtype is not torch.float32 or out_scale.get_device() != dev or out_scale.shape != want or (
                not out_scale.is_contiguous()):
            raise ValueError(f"out_scale must be a contiguous float32 tensor of shape {want} on cuda:{dev}")
        s_ptr = out_scale.data_ptr()
    elif out_scale is not None:
        raise ValueError("out_scale needs an 8-bit format")
    _on(dev, call, dep_norm_args_t(
        x.data_ptr(), r_ptr, w_ptr, ro_ptr, out.data_ptr(), s_ptr, _rows(x, "x", bf16, dev, shape), r_stride,
        ro_stride, _rows(out, "out", dtype, dev, shape), rows, cols, _QUANT[quant], eps), stream)
    return out if quant is None else (out, out_scale)


def add_rms_norm(x, weight=None, residual=None, *, eps: float = 1e-6, quant=None, out=None, out_scale=None,
                 residual_out=None, stream=None):
    """h = x + residual (stored to residual_out, by default over residual), then
    h / rms(h) * weight: BF16, or with quant="int8" / "e4m3" 8-bit values and their
    scales (see dep_add_rms_norm in include/dep_projection.h).

    x, residual: bfloat16 [rows, cols] with contiguous rows; weight: bfloat16 [cols].
    Returns out, or (out, out_scale) for an 8-bit format; both are allocated where
    omitted.  scale is [rows] (int8) or [rows, ceil(cols / 128)] (e4m3)."""
    return _norm_call(dep_add_rms_norm, x, weight, residual, residual_out, eps, quant, out, out_scale, stream)


def quantize_rows(x, *, quant="int8", out=None, out_scale=None, stream=None):
    """The rows of a bfloat16 matrix in 8 bits: (values, scales), as add_rms_norm
    stores them but without a norm."""
    if quant is None:
        raise ValueError("quant must be 'int8' or 'e4m3'")
    return _norm_call(dep_quantize_rows, x, None, None, None, 0.0, quant, out, out_scale, stream)


def _heads(t, name, dtype, index, shape):
    """Stride between the tokens of [tokens, heads, ...] whose inner dimensions are contiguous."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        strides, inner = t.stride(), shape[-1]
        if strides[-1] == 1 or inner == 1:
            if len(strides) == 2:
                return strides[0] if shape[0] > 1 else inner
            if strides[1] == inner or shape[1] == 1:
                return strides[0] if shape[0] > 1 else inner * shape[1]
    raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} with contiguous heads on cuda:{index}")


def gated_delta_rule(q, k, v, g, beta, state=None, state_out=None, *, cu_seqlens=None, n_seq: int | None = None,
                     slots=None, scale: float | None = None, l2norm: bool = False, out=None, stream=None):
    """The gated delta rule over packed sequences (see dep_delta_rule in
    include/dep_projection.h): for each token S <- S diag(exp(g)), then
    S <- S + beta (v - S k) k^T, o = scale S q.

    q, k: bfloat16 [tokens, Hq, Dk]; v: bfloat16 [tokens, Hv, Dv]; g: float32
    [tokens, Hv] or, for a decay of each key channel, [tokens, Hv, Dk]; beta:
    float32 [tokens, Hv].  Heads are contiguous, tokens any stride apart.
    cu_seqlens: int32 [n_seq + 1] on the device, or None for n_seq (default 1)
    sequences of equal length; tokens outside the table keep what out holds there
    (in a new out, anything).  state, state_out: float32 [n_states, Hv, Dv, Dk];
    state None starts from zeros, state_out defaults to state (updated in place).
    slots: int32 [n_seq] on the device, each sequence's place among the states
    (outside 0..n_states-1: padding).  scale defaults to Dk ** -0.5.  The workspace
    is the allocator's (up to 2 GiB, for sequences of eight tokens and more on
    average).  Returns out, bfloat16 [tokens, Hv, Dv] (allocated where omitted)."""
    import torch
    dev, bf16, f32 = q.get_device(), torch.bfloat16, torch.float32
    qk_shape, v_shape = q.shape, v.shape
    if len(qk_shape) != 3 or len(v_shape) != 3 or dev < 0:
        raise ValueError("q, k [tokens, Hq, Dk] and v [tokens, Hv, Dv] must be CUDA tensors of three dimensions")
    T, hq, dk = qk_shape
    _, hv, dv = v_shape
    if v_shape[0] != T:
        raise ValueError(f"v must have q's {T} tokens")
    channel = g.dim() == 3
    if state_out is None:
        state_out = state
        if state is None:
            raise ValueError("state_out must be given where state is not")
    n_states = state_out.shape[0]
    for s in (state_out,) if state is None or state is state_out else (state, state_out):
        if s.dtype is not f32 or s.get_device() != dev or s.shape != (n_states, hv, dv, dk) or not s.is_contiguous():
            raise ValueError(
                f"state and state_out must be contiguous float32 tensors [n_states, {hv}, {dv}, {dk}] on cuda:{dev}")
    if cu_seqlens is not None:
        n = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.get_device() != dev or n < 0 or (
                not cu_seqlens.is_contiguous() or (n_seq is not None and n_seq != n)):
            raise ValueError(f"cu_seqlens must be a contiguous int32 vector of n_seq + 1 on cuda:{dev}")
        n_seq = n
    elif n_seq is None:
        n_seq = 1
    if slots is not None and (slots.dtype is not torch.int32 or slots.get_device() != dev or slots.shape != (n_seq,)
                              or not slots.is_contiguous()):
        raise ValueError(f"slots must be a contiguous int32 vector of {n_seq} on cuda:{dev}")
    if out is None:
        out = _empty(v_shape, bf16, q.device, stream)
    args = dep_delta_args_t(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(state), state_out.data_ptr(),
        out.data_ptr(), _ptr(cu_seqlens), _ptr(slots), _heads(q, "q", bf16, dev, qk_shape),
        _heads(k, "k", bf16, dev, qk_shape), _heads(v, "v", bf16, dev, v_shape),
        _heads(g, "g", f32, dev, (T, hv, dk) if channel else (T, hv)), _heads(beta, "beta", f32, dev, (T, hv)),
        _heads(out, "out", bf16, dev, v_shape), T, n_states, n_seq, hq, hv, dk, dv,
        (DEP_DELTA_CHANNEL if channel else 0) | (DEP_DELTA_L2NORM if l2norm else 0),
        dk ** -0.5 if scale is None else scale)
    if T > n_seq:  # more than single tokens
        args.workspace_bytes = dep_delta_workspace(args)
        if args.workspace_bytes:
            workspace = _empty((args.workspace_bytes,), torch.uint8, q.device, stream)
            args.workspace = workspace.data_ptr()
    _on(dev, dep_delta_rule, args, stream)
    return out


class Int8Projection:
    """A TP1 linear over one resident int8 weight W[N,K] with a scale for each
    output channel: ``run(x, x_scale)`` writes
    BF16(x_scale[b] * w_scale[n] * sum_k x[b,k] W[n,k]) for int8 x with a scale for
    each row, as add_rms_norm(quant="int8") and quantize_rows make them.  Batches of
    more than max_rows rows run in passes.  One projection per stream."""

    def __init__(self, weight, weight_scale, max_rows: int = 256):
        import torch
        if weight.dtype != torch.int8 or not weight.is_cuda or weight.dim() != 2 or not weight.is_contiguous():
            raise ValueError("weight must be a contiguous CUDA int8 tensor [N, K]")
        self.N, self.K = weight.shape
        if weight_scale.dtype != torch.float32 or weight_scale.device != weight.device or (
                weight_scale.shape != (self.N,)) or not weight_scale.is_contiguous():
            raise ValueError(f"weight_scale must be a contiguous float32 vector of {self.N} on {weight.device}")
        self.weight, self.weight_scale = weight, weight_scale
        self.index = weight.get_device()
        with torch.cuda.device(self.index):
            self.plan = dep_int8_plan(self.N, self.K, max_rows)

    def run(self, x, x_scale, out=None, stream=None):
        import torch
        dev, shape = self.index, x.shape
        if x.dtype is not torch.int8 or x.get_device() != dev or len(shape) != 2 or shape[1] != self.K or (
                not x.is_contiguous()):
            raise ValueError(f"x must be a contiguous int8 tensor [rows, {self.K}] on cuda:{dev}")
        B = shape[0]
        if x_scale.dtype is not torch.float32 or x_scale.get_device() != dev or x_scale.numel() != B or (
                not x_scale.is_contiguous()):
            raise ValueError(f"x_scale must be a contiguous float32 vector of {B} on cuda:{dev}")
        if out is None:
            out = _empty((B, self.N), torch.bfloat16, x.device, stream)
        elif out.dtype is not torch.bfloat16 or out.get_device() != dev or out.shape != (B, self.N) or (
                not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous bfloat16 tensor [{B}, {self.N}] on cuda:{dev}")
        _on(dev, self._run, (x, x_scale, out, B), stream)
        return out

    def _run(self, args, stream):
        x, x_scale, out, B = args
        dep_int8_run(self.plan, x, x_scale, self.weight, self.weight_scale, out, B, stream)

    def close(self):
        if getattr(self, "plan", None):
            dep_int8_plan_destroy(self.plan)
            self.plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
