"""ctypes binding of libzero_dp.so (argument marshalling only).

Every function here converts its arguments (torch tensors or raw device
addresses, Python numbers) into the C structs of include/zero_dp.h and calls
the library; all computation happens inside the library.  If the shared
library is missing, loading raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import List, Optional, Sequence, Tuple

# the in-tree build; ZERO_DP_LIBRARY names another build of the same ABI
# (the host-only sanitizer build that the host-side tests load)
_LIB_PATH = os.environ.get("ZERO_DP_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                              "libzero_dp.so")
_lib = None

ZERO_OK = 0
ZERO_EINVAL = -1
ZERO_EALIGN = -2
ZERO_EOVERFLOW = -3
ZERO_ECAPACITY = -4
ZERO_EALIAS = -5
ZERO_EHIP = -6

EXPORTED = (
    "zero_strerror", "zero_last_hip_error", "zero_abi_version", "zero_plan_partitions",
    "zero_memory_model", "zero_workspace_bytes", "zero_reduce_owned", "zero_ctl_init",
    "zero_adam_step", "zero_adam_step_clipped", "zero_adam_step_bucket", "zero_restore_skipped",
    "zero_emit_fp16", "zero_gather_params", "zero_adam_step_noalloc", "zero_calib_triad",
    "zero_calib_stream_mix", "zero_adam_step_buckets", "zero_gather_layers", "zero_calib_slice_read",
    "zero_tensors_plan", "zero_tensors_grad_norm", "zero_tensors_adam_step", "zero_mx8_encode", "zero_mx8_decode",
)
ABI_VERSION = 7
BUCKET_FIRST = 1
BUCKET_LAST = 2


class ZeroError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().zero_strerror(status).decode()
        if status == ZERO_EHIP:
            msg += f" (hipError {lib().zero_last_hip_error()})"
        super().__init__(f"{where}: {msg} [{status}]")
        self.status = status


class Plan(C.Structure):
    _fields_ = [("psi", C.c_int64), ("nd", C.c_int32), ("align", C.c_int32), ("part", C.c_int64),
                ("padded", C.c_int64), ("pad", C.c_int64)]


class Frag(C.Structure):
    _fields_ = [("tensor", C.c_int32), ("rank", C.c_int32), ("tensor_off", C.c_int64),
                ("flat_off", C.c_int64), ("local_off", C.c_int64), ("len", C.c_int64)]


class MemReport(C.Structure):
    _fields_ = [(k, C.c_double) for k in ("params_bytes", "grads_bytes", "optim_bytes", "total_bytes",
                                          "comm_elems", "comm_elems_ring", "reduction_vs_dp")]


class GradSrc(C.Structure):
    _fields_ = [("base", C.c_void_p), ("slice_stride", C.c_int64), ("elem_off", C.c_int64),
                ("n", C.c_int64), ("nd", C.c_int32), ("reserved", C.c_int32), ("loss_scale", C.c_double)]


class StepCtl(C.Structure):
    _fields_ = [("cur", C.c_int32), ("t", C.c_int32), ("overflow", C.c_int32), ("good_steps", C.c_int32),
                ("beta1_pow", C.c_double), ("beta2_pow", C.c_double), ("sumsq", C.c_double),
                ("skipped", C.c_int64), ("loss_scale", C.c_double), ("clip_coef", C.c_double)]


class Bucket(C.Structure):
    _fields_ = [("src", GradSrc), ("win_off", C.c_int64)]


MAX_BUCKETS_PER_CALL = 1024
MX8_BLOCK = 32
TYPE_NONE, TYPE_F32, TYPE_F16, TYPE_BF16, TYPE_MX8 = range(5)
ROUNDING = {"nearest": 0, "stochastic": 1}


class Tensor(C.Structure):
    _fields_ = [(k, C.c_void_p) for k in ("master", "grad", "param", "exp_avg", "exp_avg_sq", "avg_scale",
                                          "sq_scale")] + \
               [("n", C.c_int64), ("flat_off", C.c_int64), ("reserved", C.c_int64)]


class TensorListInfo(C.Structure):
    _fields_ = [(k, C.c_int32) for k in ("n_tensors", "grad_type", "param_type", "state_type")] + \
               [(k, C.c_int64) for k in ("n_elems", "n_chunks", "table_bytes", "reserved")]


class AdamState(C.Structure):
    _fields_ = [("master", C.c_void_p * 2), ("exp_avg", C.c_void_p * 2), ("exp_avg_sq", C.c_void_p * 2),
                ("ctl", C.c_void_p)]


class AdamHp(C.Structure):
    _fields_ = [(k, C.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay", "max_grad_norm",
                                          "scale_growth", "scale_backoff")] + \
               [("scale_interval", C.c_int32), ("reserved", C.c_int32)]


def lib():
    """Loads libzero_dp.so from the package directory (raises if absent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run "
                           "`python -m zero_partitioned_mixed_buffer_amd.build_lib`")
    # torch first: the library's libamdhip64.so.7 then resolves to the HIP
    # runtime torch has loaded, and the process holds one HIP runtime.
    # Loaded the other way round, torch loads a second copy of its own and
    # the library's runtime reports no device.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = C.CDLL(_LIB_PATH)
    P = C.c_void_p
    L.zero_strerror.restype = C.c_char_p
    L.zero_strerror.argtypes = [C.c_int]
    L.zero_last_hip_error.restype = C.c_int
    L.zero_abi_version.restype = C.c_int
    L.zero_plan_partitions.argtypes = [C.POINTER(C.c_int64), C.c_int32, C.c_int32, C.c_int32,
                                       C.POINTER(Plan), C.POINTER(Frag), C.c_int64, C.POINTER(C.c_int64)]
    L.zero_memory_model.argtypes = [C.c_double, C.c_int32, C.c_int32, C.c_int32, C.POINTER(MemReport)]
    L.zero_workspace_bytes.restype = C.c_int64
    L.zero_reduce_owned.argtypes = [C.POINTER(GradSrc), P, P, P, P, P]
    L.zero_ctl_init.argtypes = [C.POINTER(StepCtl), C.c_double]
    L.zero_ctl_init.restype = None
    L.zero_adam_step.argtypes = [C.POINTER(GradSrc), C.POINTER(AdamState), C.POINTER(AdamHp), P,
                                 C.c_int64, P, P]
    L.zero_adam_step_noalloc.argtypes = [C.POINTER(GradSrc), C.POINTER(AdamState), C.POINTER(AdamHp), P,
                                         C.c_int64, P]
    L.zero_adam_step_clipped.argtypes = [C.POINTER(GradSrc), C.POINTER(AdamState), C.POINTER(AdamHp), P, P,
                                         C.c_int64, P, P]
    L.zero_adam_step_bucket.argtypes = [C.POINTER(GradSrc), C.POINTER(AdamState), C.POINTER(AdamHp), C.c_int64,
                                        C.c_int64, P, C.c_int64, C.c_int32, P, P]
    L.zero_restore_skipped.argtypes = [C.POINTER(AdamState), C.c_int64, P, C.c_int64, P]
    L.zero_emit_fp16.argtypes = [P, C.c_int64, P, C.c_int64, P]
    L.zero_gather_params.argtypes = [C.POINTER(C.c_void_p), C.c_int32, C.c_int64, C.c_int64, C.c_int64, P, P]
    L.zero_adam_step_buckets.argtypes = [C.POINTER(Bucket), C.c_int32, C.POINTER(AdamState), C.POINTER(AdamHp),
                                         C.c_int64, P, C.c_int64, C.c_int32, P, P]
    L.zero_gather_layers.argtypes = [C.POINTER(C.c_void_p), C.c_int32, C.c_int64, C.POINTER(C.c_int64), C.c_int32,
                                     C.POINTER(C.c_void_p), P]
    L.zero_calib_triad.argtypes = [P, P, P, C.c_float, C.c_int64, P]
    L.zero_calib_stream_mix.argtypes = [C.POINTER(GradSrc), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), P, P]
    L.zero_calib_slice_read.argtypes = [C.POINTER(GradSrc), P, P]
    L.zero_tensors_plan.argtypes = [C.POINTER(Tensor), C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                    C.POINTER(TensorListInfo), P, C.c_int64]
    L.zero_tensors_grad_norm.argtypes = [C.POINTER(TensorListInfo), P, C.c_double, P, P, P, P, P]
    L.zero_tensors_adam_step.argtypes = [C.POINTER(TensorListInfo), P, C.POINTER(AdamHp), C.c_double, P, P, P,
                                         C.c_int32, C.c_uint64, P, P]
    L.zero_mx8_encode.argtypes = [P, C.c_int64, C.c_int32, P, P, C.c_int32, C.c_uint64, C.c_int64, C.c_int64, P]
    L.zero_mx8_decode.argtypes = [P, P, C.c_int64, C.c_int32, P, P]
    for name in ("zero_tensors_plan", "zero_tensors_grad_norm", "zero_tensors_adam_step", "zero_mx8_encode",
                 "zero_mx8_decode", "zero_plan_partitions", "zero_memory_model", "zero_reduce_owned", "zero_adam_step",
                 "zero_adam_step_noalloc", "zero_calib_triad", "zero_calib_stream_mix", "zero_adam_step_buckets",
                 "zero_gather_layers", "zero_calib_slice_read",
                 "zero_adam_step_clipped", "zero_adam_step_bucket", "zero_restore_skipped", "zero_emit_fp16",
                 "zero_gather_params"):
        getattr(L, name).restype = C.c_int
    if L.zero_abi_version() != ABI_VERSION:
        raise RuntimeError("libzero_dp.so ABI version mismatch")
    _lib = L
    return L


def _check(status: int, where: str):
    if status != ZERO_OK:
        raise ZeroError(status, where)


def _ptr(x) -> Optional[int]:
    """Device or host address of a torch tensor, or an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _is_tensor(x) -> bool:
    return x is not None and not isinstance(x, int)


_DTYPE_NAMES: dict = {}


def _dtype_name(t) -> str:
    d = t.dtype
    name = _DTYPE_NAMES.get(d)
    if name is None:
        name = _DTYPE_NAMES[d] = str(d).replace("torch.", "")
    return name


def _check_span(t, off: int, n: int, kinds: Tuple[str, ...], what: str):
    """For a torch tensor argument: dtype one of ``kinds``, elements laid out
    contiguously, [off, off + n) inside the tensor, on a GPU.  Raw addresses
    (ints) and None pass through (the library checks what it can)."""
    if t is None or isinstance(t, int):
        return
    if _dtype_name(t) not in kinds:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {kinds}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if off < 0 or n < 0 or off + n > t.numel():
        raise ValueError(f"{what}: elements [{off}, {off + n}) outside a tensor of {t.numel()}")
    if not t.is_cuda:
        raise ValueError(f"{what}: must be a device tensor")


_F16 = ("float16", "int16")


def _check_ws(ws):
    if ws is not None and not isinstance(ws, int) and (ws.numel() * ws.element_size() < workspace_bytes()
                                                      or not ws.is_cuda):
        raise ValueError(f"workspace: a device tensor of at least {workspace_bytes()} bytes")


_raw_stream = None


def _stream(stream) -> Optional[int]:
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            torch.cuda.init()
            current, raw = torch.cuda.current_device, getattr(torch._C, "_cuda_getCurrentRawStream", None)
            # the stream's address alone: 0.3 us where a Stream object takes 3
            _raw_stream = (lambda: raw(current())) if raw else \
                (lambda: int(torch.cuda.current_stream().cuda_stream))
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# ------------------------------------------------------------------ host calls
def plan_partitions(numels: Sequence[int], nd: int, align: int = 256) -> Tuple[dict, List[tuple]]:
    L = lib()
    arr = (C.c_int64 * max(len(numels), 1))(*[int(x) for x in numels])
    plan = Plan()
    n = C.c_int64(0)
    st = L.zero_plan_partitions(arr, len(numels), nd, align, C.byref(plan), None, 0, C.byref(n))
    frags: List[tuple] = []
    if st == ZERO_ECAPACITY or (st == ZERO_OK and n.value > 0):
        buf = (Frag * n.value)()
        st = L.zero_plan_partitions(arr, len(numels), nd, align, C.byref(plan), buf, n.value, C.byref(n))
        frags = [(f.tensor, f.rank, f.tensor_off, f.flat_off, f.local_off, f.len) for f in buf]
    _check(st, "zero_plan_partitions")
    return ({"psi": plan.psi, "nd": plan.nd, "align": plan.align, "part": plan.part,
             "padded": plan.padded, "pad": plan.pad}, frags)


def memory_model(psi: float, nd: int, stage: int, k: int = 12) -> dict:
    r = MemReport()
    _check(lib().zero_memory_model(float(psi), nd, stage, k, C.byref(r)), "zero_memory_model")
    return {name: getattr(r, name) for name, _ in MemReport._fields_}


_ws_bytes: Optional[int] = None


def workspace_bytes() -> int:
    global _ws_bytes
    if _ws_bytes is None:
        _ws_bytes = int(lib().zero_workspace_bytes())
    return _ws_bytes


def ctl_init_bytes(loss_scale: float = 65536.0) -> bytes:
    c = StepCtl()
    lib().zero_ctl_init(C.byref(c), float(loss_scale))
    return bytes(c)


def ctl_from_bytes(b: bytes) -> dict:
    c = StepCtl.from_buffer_copy(b)
    return {name: getattr(c, name) for name, _ in StepCtl._fields_}


def ctl_to_bytes(fields: dict) -> bytes:
    """The control block's bytes from its fields (the inverse of ctl_from_bytes)."""
    c = StepCtl()
    for name, _ in StepCtl._fields_:
        setattr(c, name, fields[name])
    return bytes(c)


CTL_BYTES = C.sizeof(StepCtl)


# ------------------------------------------------------------------ device calls
def grad_src(base, slice_stride: int, elem_off: int, n: int, nd: int, loss_scale: float) -> GradSrc:
    """Gradient source: slice k of the window is base[k, elem_off:elem_off+n].
    A torch ``base`` must be a 2-D fp16 device tensor whose rows are
    ``slice_stride`` elements apart and that holds the whole window."""
    if _is_tensor(base):
        if _dtype_name(base) not in _F16:
            raise ValueError(f"gradient slices: dtype {base.dtype}, expected float16")
        if base.dim() != 2 or base.stride(1) != 1:
            raise ValueError("gradient slices: a 2-D tensor [Nd, stride] with unit element stride")
        if base.shape[0] < nd or (nd > 1 and base.stride(0) != slice_stride):
            raise ValueError(f"gradient slices: {base.shape[0]} rows {base.stride(0)} apart, "
                             f"expected {nd} rows {slice_stride} apart")
        if elem_off < 0 or n < 0 or elem_off + n > base.shape[1]:
            raise ValueError(f"gradient slices: columns [{elem_off}, {elem_off + n}) outside {base.shape[1]}")
        if not base.is_cuda:
            raise ValueError("gradient slices: must be a device tensor")
    return GradSrc(_ptr(base), int(slice_stride), int(elem_off), int(n), int(nd), 0, float(loss_scale))


def adam_state(master: Sequence, exp_avg: Sequence, exp_avg_sq: Sequence, ctl) -> AdamState:
    """Ping-pong state; with torch tensors, each a contiguous fp32 device
    array, and the steps then check that the window fits in all six."""
    s = AdamState()
    arrays = [*master, *exp_avg, *exp_avg_sq]
    for a in arrays:
        _check_span(a, 0, 0, ("float32",), "state array")
    for i in range(2):
        s.master[i] = _ptr(master[i])
        s.exp_avg[i] = _ptr(exp_avg[i])
        s.exp_avg_sq[i] = _ptr(exp_avg_sq[i])
    if _is_tensor(ctl) and (ctl.numel() * ctl.element_size() < CTL_BYTES or not ctl.is_cuda):
        raise ValueError(f"control block: a device tensor of at least {CTL_BYTES} bytes")
    s.ctl = _ptr(ctl)
    if all(_is_tensor(a) for a in arrays):
        s._numel = min(int(a.numel()) for a in arrays)
    return s


def _check_state(state: AdamState, n: int):
    cap = getattr(state, "_numel", None)
    if cap is not None and n > cap:
        raise ValueError(f"state arrays of {cap} elements cannot hold a window of {n}")


def adam_hp(lr: float, beta1: float, beta2: float, eps: float, weight_decay: float,
            max_grad_norm: float = 0.0, scale_interval: int = 0, scale_growth: float = 2.0,
            scale_backoff: float = 0.5) -> AdamHp:
    return AdamHp(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                  float(max_grad_norm), float(scale_growth), float(scale_backoff), int(scale_interval), 0)


def reduce_owned(src: GradSrc, grad_out, overflow, sumsq, workspace, stream=None):
    _check_span(grad_out, 0, src.n, ("float32",), "gradient output")
    _check_span(overflow, 0, 1, ("int32",), "overflow flag")
    _check_span(sumsq, 0, 1, ("float64",), "sum of squares")
    _check_ws(workspace)
    _check(lib().zero_reduce_owned(C.byref(src), _ptr(grad_out), _ptr(overflow), _ptr(sumsq),
                                   _ptr(workspace), _stream(stream)), "zero_reduce_owned")


def adam_step(src: GradSrc, state: AdamState, hp: AdamHp, allgather, allgather_off: int, workspace,
              stream=None):
    _check_state(state, src.n)
    _check_span(allgather, allgather_off, src.n, _F16, "all-gather buffer")
    _check_ws(workspace)
    _check(lib().zero_adam_step(C.byref(src), C.byref(state), C.byref(hp), _ptr(allgather),
                                int(allgather_off), _ptr(workspace), _stream(stream)), "zero_adam_step")


def adam_step_noalloc(src: GradSrc, state: AdamState, hp: AdamHp, allgather, allgather_off: int, stream=None):
    """zero_adam_step on the library's own per-GPU scratch (no workspace)."""
    _check_state(state, src.n)
    _check_span(allgather, allgather_off, src.n, _F16, "all-gather buffer")
    _check(lib().zero_adam_step_noalloc(C.byref(src), C.byref(state), C.byref(hp), _ptr(allgather),
                                        int(allgather_off), _stream(stream)), "zero_adam_step_noalloc")


def adam_step_clipped(src: GradSrc, state: AdamState, hp: AdamHp, grad_buf, allgather, allgather_off: int,
                      workspace, stream=None):
    _check_state(state, src.n)
    _check_span(grad_buf, 0, src.n, ("float32",), "gradient buffer")
    _check_span(allgather, allgather_off, src.n, _F16, "all-gather buffer")
    _check_ws(workspace)
    _check(lib().zero_adam_step_clipped(C.byref(src), C.byref(state), C.byref(hp), _ptr(grad_buf),
                                        _ptr(allgather), int(allgather_off), _ptr(workspace), _stream(stream)),
           "zero_adam_step_clipped")


def adam_step_bucket(src: GradSrc, state: AdamState, hp: AdamHp, win_off: int, window_n: int, allgather,
                     allgather_off: int, phase: int, workspace, stream=None):
    _check_state(state, window_n)
    _check_span(allgather, allgather_off, window_n, _F16, "all-gather buffer")
    _check_ws(workspace)
    _check(lib().zero_adam_step_bucket(C.byref(src), C.byref(state), C.byref(hp), int(win_off), int(window_n),
                                       _ptr(allgather), int(allgather_off), int(phase), _ptr(workspace),
                                       _stream(stream)), "zero_adam_step_bucket")


def bucket_array(buckets: Sequence[Tuple[GradSrc, int]]):
    """The zero_bucket array of (gradient source, window offset) pairs, for
    callers that pass the same buckets step after step."""
    return (Bucket * max(len(buckets), 1))(*[Bucket(src, int(off)) for src, off in buckets]), len(buckets)


def adam_step_buckets(buckets, state: AdamState, hp: AdamHp, window_n: int,
                      allgather, allgather_off: int, phase: int, workspace, stream=None):
    """Several arrived buckets of a bucketed step in one call: ``buckets``
    lists (gradient source, window offset) pairs, or is what bucket_array
    made of such a list."""
    _check_state(state, window_n)
    _check_span(allgather, allgather_off, window_n, _F16, "all-gather buffer")
    _check_ws(workspace)
    arr, nb = buckets if isinstance(buckets, tuple) else bucket_array(buckets)
    _check(lib().zero_adam_step_buckets(arr, nb, C.byref(state), C.byref(hp), int(window_n),
                                        _ptr(allgather), int(allgather_off), int(phase), _ptr(workspace),
                                        _stream(stream)), "zero_adam_step_buckets")


def restore_skipped(state: AdamState, n: int, allgather, allgather_off: int, stream=None):
    _check_state(state, n)
    _check_span(allgather, allgather_off, n, _F16, "all-gather buffer")
    _check(lib().zero_restore_skipped(C.byref(state), int(n), _ptr(allgather), int(allgather_off),
                                      _stream(stream)), "zero_restore_skipped")


def emit_fp16(master, n: int, allgather, allgather_off: int, stream=None):
    _check_span(master, 0, n, ("float32",), "master")
    _check_span(allgather, allgather_off, n, _F16, "all-gather buffer")
    _check(lib().zero_emit_fp16(_ptr(master), int(n), _ptr(allgather), int(allgather_off),
                                _stream(stream)), "zero_emit_fp16")


def gather_params(windows: Sequence, part: int, lo: int, hi: int, dst, stream=None):
    """Flat elements [lo, hi) of the partitioned fp16 parameters into dst;
    ``windows`` lists the Nd owners' windows (tensors, addresses or None)."""
    if part > 0 and hi > lo:  # the windows the range touches (the library rejects a null one)
        for w in windows[max(lo, 0) // part:min((hi - 1) // part + 1, len(windows))]:
            _check_span(w, 0, part, _F16, "parameter window")
    _check_span(dst, 0, max(hi - lo, 0), _F16, "layer buffer")
    arr = (C.c_void_p * max(len(windows), 1))(*[_ptr(w) for w in windows])
    _check(lib().zero_gather_params(arr, len(windows), int(part), int(lo), int(hi), _ptr(dst), _stream(stream)),
           "zero_gather_params")


def gather_layers(windows: Sequence, part: int, ranges: Sequence[Tuple[int, int]], dsts: Sequence, stream=None):
    """Flat ranges [lo, hi) of the partitioned fp16 parameters, range q into
    dsts[q], with the ranges' pieces sharing launches."""
    for (lo, hi), d in zip(ranges, dsts):
        if part > 0 and hi > lo:
            for w in windows[max(lo, 0) // part:min((hi - 1) // part + 1, len(windows))]:
                _check_span(w, 0, part, _F16, "parameter window")
        _check_span(d, 0, max(hi - lo, 0), _F16, "layer buffer")
    if len(ranges) != len(dsts):
        raise ValueError("one destination per range")
    arr = (C.c_void_p * max(len(windows), 1))(*[_ptr(w) for w in windows])
    rng = (C.c_int64 * max(2 * len(ranges), 1))(*[int(x) for r in ranges for x in r])
    dst = (C.c_void_p * max(len(dsts), 1))(*[_ptr(d) for d in dsts])
    _check(lib().zero_gather_layers(arr, len(windows), int(part), rng, len(ranges), dst, _stream(stream)),
           "zero_gather_layers")


# ----------------------------------------------------------------- tensor lists
_LIST_TYPES = {"float32": TYPE_F32, "float16": TYPE_F16, "bfloat16": TYPE_BF16}
_CODES = ("float8_e4m3fn", "uint8")
_SCALES = ("float8_e8m0fnu", "uint8")


def _check_current(t, what: str, cur: Optional[int] = None):
    """A tensor of the current device: the launch goes to that device's stream."""
    if _is_tensor(t):
        if not t.is_cuda:
            raise ValueError(f"{what}: must be a device tensor")
        if cur is None:
            import torch
            cur = torch.cuda.current_device()
        if t.get_device() != cur:
            raise ValueError(f"{what}: on {t.device}, but the current device is {cur}")


def _check_operand(t, n: int, kinds: Tuple[str, ...], what: str, cur: int):
    """_check_span from element 0 and _check_current."""
    if _is_tensor(t) and not (_dtype_name(t) in kinds and t.numel() >= n and t.get_device() == cur
                              and t.is_contiguous()):
        _check_span(t, 0, n, kinds, what)
        _check_current(t, what, cur)


def _current_device() -> int:
    import torch
    return torch.cuda.current_device()


def _column(tensors: Sequence, numels: Sequence[int], kinds: Tuple[str, ...], what: str,
            per: int = 1) -> Tuple[str, List[int]]:
    """Checks a list's tensors of one kind (one dtype, contiguous, one
    element for ``per`` of the list's) and returns the dtype's name and the
    addresses."""
    import torch
    if len(tensors) != len(numels):
        raise ValueError(f"{what}: {len(tensors)} entries for {len(numels)} gradients")
    if not all(isinstance(t, torch.Tensor) for t in tensors):
        raise ValueError(f"{what}: torch tensors expected")
    names = {_DTYPE_NAMES.get(d) or str(d).replace("torch.", "") for d in {t.dtype for t in tensors}}
    if len(names) > 1 or not names <= set(kinds):
        raise ValueError(f"{what}: one dtype of {kinds} expected, got {sorted(names)}")
    for t, n in zip(tensors, numels):
        if t.numel() != -(-n // per):
            raise ValueError(f"{what}: {t.numel()} elements where {-(-n // per)} are expected")
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensors must be contiguous")
    return names.pop() if names else kinds[0], [t.data_ptr() for t in tensors]


def _on_current(columns: Sequence[Sequence]):
    """Every tensor of the columns is on the current device."""
    cur = -1
    for col in columns:
        for t in col:
            d = t.get_device()
            if d != cur or d < 0:
                _check_current(t, "tensor list")
                cur = d


def _grad_column(grads: Sequence) -> Tuple[int, List[int], List[int]]:
    import torch
    numels = [int(t.numel()) if isinstance(t, torch.Tensor) else 0 for t in grads]
    name, ptrs = _column(grads, numels, tuple(_LIST_TYPES), "gradients")
    return _LIST_TYPES[name], ptrs, numels


class TensorList:
    """A planned list of tensors: its table in device memory, and the tensors
    it points to (kept alive here).  Made by tensor_list().  ``written``:
    those of the tensors that a step writes and that require gradients."""

    def __init__(self, info: TensorListInfo, table, tensors, written=()):
        self.info = info
        self.ref = C.byref(info)
        self.table = table
        self.tensors = tensors
        self.written = [t for t in written if t.requires_grad]
        self.numel = int(info.n_elems)

    def count_write(self):
        """Tells autograd of a step: a backward pass through a graph that has
        saved one of the weights before it raises."""
        if self.written:
            from torch.autograd.graph import increment_version
            increment_version(self.written)


def tensor_list(grads: Sequence, masters: Optional[Sequence] = None, params: Optional[Sequence] = None,
                exp_avg: Optional[Sequence] = None, exp_avg_sq: Optional[Sequence] = None,
                avg_scale: Optional[Sequence] = None, sq_scale: Optional[Sequence] = None,
                flat_offs: Optional[Sequence[int]] = None) -> TensorList:
    """Plans a list of torch tensors on the current device (zero_tensors_plan)
    and uploads its table.

    ``grads`` alone makes a list for norms.  A list for steps has as many
    ``masters`` (float32), ``exp_avg`` and ``exp_avg_sq`` (float32; or e4m3
    codes, and then ``avg_scale`` and ``sq_scale`` with one byte for 32
    elements), and may have 16-bit ``params``.  Every tensor is contiguous,
    and the list holds their addresses: plan again when one moves.
    ``flat_offs`` are the tensors' first random counters (default: packed in
    list order)."""
    steps = masters is not None
    if any((v is not None) != steps for v in (exp_avg, exp_avg_sq)):
        raise ValueError("masters, exp_avg and exp_avg_sq come together")
    if not steps and (params is not None or avg_scale is not None or sq_scale is not None):
        raise ValueError("a list of gradients alone has no params and no scales")
    gtype, gptr, numels = _grad_column(grads)
    ptype = stype = TYPE_NONE
    columns, keep = {"grad": gptr}, [list(grads)]
    if steps:
        _, columns["master"] = _column(masters, numels, ("float32",), "masters")
        if params is not None:
            name, columns["param"] = _column(params, numels, ("float16", "bfloat16"), "params")
            ptype = _LIST_TYPES[name]
        kind, columns["exp_avg"] = _column(exp_avg, numels, ("float32", *_CODES), "exp_avg")
        stype = TYPE_F32 if kind == "float32" else TYPE_MX8
        _, columns["exp_avg_sq"] = _column(exp_avg_sq, numels, (kind,), "exp_avg_sq")
        if (stype == TYPE_MX8) != (avg_scale is not None) or (stype == TYPE_MX8) != (sq_scale is not None):
            raise ValueError("states in 8 bits, and no others, come with avg_scale and sq_scale")
        if stype == TYPE_MX8:
            _, columns["avg_scale"] = _column(avg_scale, numels, _SCALES, "avg_scale", MX8_BLOCK)
            _, columns["sq_scale"] = _column(sq_scale, numels, _SCALES, "sq_scale", MX8_BLOCK)
        keep += [list(c) for c in (masters, params, exp_avg, exp_avg_sq, avg_scale, sq_scale) if c is not None]
    _on_current(keep)
    return _plan_list(numels, columns, gtype, ptype, stype, flat_offs, keep, (*(masters or ()), *(params or ())))


def _plan_list(numels: Sequence[int], columns: dict, gtype: int, ptype: int, stype: int,
               flat_offs: Optional[Sequence[int]], keep, written=()) -> TensorList:
    """The list of tensors at the addresses in ``columns`` (zero_tensor's
    fields), its table uploaded to the current device."""
    import numpy as np
    import torch
    count = len(numels)
    if flat_offs is not None and len(flat_offs) != count:
        raise ValueError(f"flat_offs: {len(flat_offs)} entries for {count} gradients")
    arr = np.zeros((max(count, 1), len(Tensor._fields_)), dtype=np.int64)
    at = {name: i for i, (name, _) in enumerate(Tensor._fields_)}
    if count:
        arr[:, at["n"]] = numels
        arr[:, at["flat_off"]] = np.concatenate([[0], np.cumsum(numels[:-1])]) if flat_offs is None else flat_offs
        for name, ptrs in columns.items():
            arr[:, at[name]] = ptrs
    tensors = arr.ctypes.data_as(C.POINTER(Tensor))
    info = TensorListInfo()
    st = lib().zero_tensors_plan(tensors, count, gtype, ptype, stype, C.byref(info), None, 0)
    if st not in (ZERO_OK, ZERO_ECAPACITY):
        _check(st, "zero_tensors_plan")
    if info.table_bytes == 0:
        return TensorList(info, None, keep, written)
    host = torch.empty(int(info.table_bytes) + 16, dtype=torch.uint8)
    host = host[-host.data_ptr() % 16:][:int(info.table_bytes)]
    _check(lib().zero_tensors_plan(tensors, count, gtype, ptype, stype, C.byref(info), host.data_ptr(), host.numel()),
           "zero_tensors_plan")
    return TensorList(info, host.to(torch.device("cuda", torch.cuda.current_device())), keep, written)


def tensors_grad_norm(lst: TensorList, overflow, sumsq, workspace, loss_scale: float = 1.0, ctl=None, stream=None):
    """sum g^2 of the list's gradients over ``loss_scale`` (or the control
    block's scale) into ``sumsq``, and whether it is not finite into ``overflow``."""
    cur = _current_device()
    _check_operand(overflow, 1, ("int32",), "overflow flag", cur)
    _check_operand(sumsq, 1, ("float64",), "sum of squares", cur)
    _check_ws(workspace)
    for t, what in ((workspace, "workspace"), (ctl, "control block"), (lst.table, "tensor list")):
        _check_current(t, what, cur)
    _check_ctl(ctl)
    _check(lib().zero_tensors_grad_norm(lst.ref, _ptr(lst.table), float(loss_scale), _ptr(ctl),
                                        _ptr(overflow), _ptr(sumsq), _ptr(workspace), _stream(stream)),
           "zero_tensors_grad_norm")


def _check_ctl(ctl):
    if _is_tensor(ctl) and (ctl.numel() * ctl.element_size() < CTL_BYTES or not ctl.is_cuda):
        raise ValueError(f"control block: a device tensor of at least {CTL_BYTES} bytes")


def _rounding(name: str) -> int:
    if name not in ROUNDING:
        raise ValueError(f"rounding: {name!r}, expected one of {tuple(ROUNDING)}")
    return ROUNDING[name]


def tensors_adam_step(lst: TensorList, hp: AdamHp, ctl, workspace, loss_scale: float = 1.0, overflow=None,
                      sumsq=None, rounding: str = "nearest", seed: int = 0, stream=None):
    """One Adam/AdamW step of every tensor of the list, in place.  Weights and
    copies that required gradients when the list was made count it as torch's
    in-place operations do (skipped steps too; a graph's replays do not)."""
    cur = _current_device()
    _check_operand(overflow, 1, ("int32",), "overflow flag", cur)
    _check_operand(sumsq, 1, ("float64",), "sum of squares", cur)
    _check_ws(workspace)
    for t, what in ((workspace, "workspace"), (ctl, "control block"), (lst.table, "tensor list")):
        _check_current(t, what, cur)
    _check_ctl(ctl)
    _check(lib().zero_tensors_adam_step(lst.ref, _ptr(lst.table), C.byref(hp), float(loss_scale),
                                        _ptr(ctl), _ptr(overflow), _ptr(sumsq), _rounding(rounding),
                                        int(seed) & (2**64 - 1), _ptr(workspace), _stream(stream)),
           "zero_tensors_adam_step")
    lst.count_write()


def _check_mx8(x, codes, scales):
    n = int(x.numel())
    cur = _current_device()
    _check_operand(x, n, ("float32",), "array", cur)
    _check_operand(codes, n, _CODES, "codes", cur)
    _check_operand(scales, -(-n // MX8_BLOCK), _SCALES, "scales", cur)
    return n


def mx8_encode(x, codes, scales, root: bool = False, rounding: str = "stochastic", seed: int = 0, step: int = 0,
               flat_off: int = 0, stream=None):
    """A float32 tensor into 8-bit blocks: its values, or their square roots."""
    n = _check_mx8(x, codes, scales)
    _check(lib().zero_mx8_encode(_ptr(x), n, int(bool(root)), _ptr(codes), _ptr(scales), _rounding(rounding),
                                 int(seed) & (2**64 - 1), int(step), int(flat_off), _stream(stream)),
           "zero_mx8_encode")


def mx8_decode(codes, scales, x, root: bool = False, stream=None):
    """8-bit blocks into a float32 tensor: the values, or their squares."""
    n = _check_mx8(x, codes, scales)
    _check(lib().zero_mx8_decode(_ptr(codes), _ptr(scales), n, int(bool(root)), _ptr(x), _stream(stream)),
           "zero_mx8_decode")


# ------------------------------------------------------------------ calibration
def calib_triad(a, b, c, q: float, n: int, stream=None):
    """a[i] = b[i] + q * c[i] over n fp32 elements (STREAM's triad)."""
    for t, what in ((a, "a"), (b, "b"), (c, "c")):
        _check_span(t, 0, n, ("float32",), f"triad {what}")
    _check(lib().zero_calib_triad(_ptr(a), _ptr(b), _ptr(c), float(q), int(n), _stream(stream)),
           "zero_calib_triad")


def calib_stream_mix(src: GradSrc, ins: Sequence, outs: Sequence, out16, stream=None):
    """The fused step's streams with no arithmetic: src's slices and ins[0..2]
    read, outs[0..2] and out16 written, src.n elements each."""
    for t in (*ins, *outs):
        _check_span(t, 0, src.n, ("float32",), "stream-mix array")
    _check_span(out16, 0, src.n, _F16, "stream-mix fp16 output")
    pin = (C.c_void_p * 3)(*[_ptr(t) for t in ins])
    pout = (C.c_void_p * 3)(*[_ptr(t) for t in outs])
    _check(lib().zero_calib_stream_mix(C.byref(src), pin, pout, _ptr(out16), _stream(stream)),
           "zero_calib_stream_mix")


def calib_slice_read(src: GradSrc, sink, stream=None):
    """src's Nd slices read alone in the fused step's schedule; the XOR fold
    of the words read is XORed into sink (a device int32/uint32 word)."""
    if sink is not None and not isinstance(sink, int):
        if _dtype_name(sink) not in ("int32", "uint32") or sink.numel() < 1 or not sink.is_cuda:
            raise ValueError("slice-read sink: one device int32 word expected")
    _check(lib().zero_calib_slice_read(C.byref(src), _ptr(sink), _stream(stream)), "zero_calib_slice_read")
