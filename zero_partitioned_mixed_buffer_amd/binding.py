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
    "zero_block8_encode", "zero_rms_norm8", "zero_rms_norm8_backward", "zero_rms_norm8_workspace_bytes",
    "zero_block8_product", "zero_block8_workspace_bytes",
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
BLOCK8 = 128
BLOCKS = {"rows": 0, "tiles": 1}
TYPE_NONE, TYPE_F32, TYPE_F16, TYPE_BF16, TYPE_MX8 = range(5)
ROUNDING = {"nearest": 0, "stochastic": 1}


class Tensor(C.Structure):
    _fields_ = [(k, C.c_void_p) for k in ("master", "grad", "param", "exp_avg", "exp_avg_sq", "avg_scale",
                                          "sq_scale")] + \
               [("n", C.c_int64), ("flat_off", C.c_int64), ("reserved", C.c_int64)]


class TensorListInfo(C.Structure):
    _fields_ = [(k, C.c_int32) for k in ("n_tensors", "grad_type", "param_type", "state_type")] + \
               [(k, C.c_int64) for k in ("n_elems", "n_chunks", "table_bytes", "reserved")]


class Matrix(C.Structure):
    _fields_ = [("data", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64), ("stride", C.c_int64),
                ("type", C.c_int32), ("reserved", C.c_int32)]


class Block8(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64),
                ("codes_stride", C.c_int64), ("scales_stride", C.c_int64), ("blocks", C.c_int32),
                ("reserved", C.c_int32)]


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
    M, M8 = C.POINTER(Matrix), C.POINTER(Block8)
    L.zero_block8_encode.argtypes = [M, P, P, C.c_int32, M8, M8, P]
    L.zero_rms_norm8.argtypes = [M, M, P, C.c_int32, C.c_double, M, M8, P, P]
    L.zero_rms_norm8_backward.argtypes = [M, M, P, C.c_int32, P, M, M, P, P, P]
    L.zero_rms_norm8_workspace_bytes.argtypes = [C.c_int64, C.c_int64]
    L.zero_block8_product.argtypes = [M8, M8, M, M, P, P]
    L.zero_block8_workspace_bytes.argtypes = [C.c_int64, C.c_int64, C.c_int64]
    for name in ("zero_rms_norm8_workspace_bytes", "zero_block8_workspace_bytes"):
        getattr(L, name).restype = C.c_int64
    for name in ("zero_block8_encode", "zero_rms_norm8", "zero_rms_norm8_backward", "zero_block8_product",
                 "zero_tensors_plan", "zero_tensors_grad_norm", "zero_tensors_adam_step", "zero_mx8_encode",
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
_raw_stream_of = None


def _stream_on(cur: int, stream) -> Optional[int]:
    """_stream, where the current device is known already."""
    global _raw_stream_of
    if stream is None:
        if _raw_stream_of is None:
            import torch
            torch.cuda.init()
            _raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: _stream(None))
        return _raw_stream_of(cur)
    return _stream(stream)


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


_get_device = None


def _current_device() -> int:
    global _get_device
    if _get_device is None:
        import torch
        _get_device = torch.cuda.current_device
    return _get_device()


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


# ------------------------------------------------------- 8-bit layer operators
# Forward and backward passes are calls of their own on the caller's buffers.
# Autograd records none of them, so a tensor that requires a gradient is refused
# where torch records (its gradient would be missing without a word); inside an
# autograd.Function or torch.no_grad() nothing is recorded and all are taken.
# Autograd sees what the calls write (_written).
# torch dtypes of the operators' tensors, filled with the first call: dtype -> ZERO_TYPE_*
_matrix_types: dict = {}
_code_types: set = set()
_scale_types: set = set()


def _fill_types():
    import torch
    _code_types.update(getattr(torch, k) for k in _CODES)
    _scale_types.update(getattr(torch, k) for k in _SCALES)
    _matrix_types.update({getattr(torch, k): v for k, v in _LIST_TYPES.items()})


_grad_enabled = None


def _refuse_grad(t, what: str):
    """For a tensor that requires a gradient: raises where torch records."""
    global _grad_enabled
    if _grad_enabled is None:
        import torch
        _grad_enabled = torch.is_grad_enabled
    if _grad_enabled():
        raise ValueError(f"{what}: the tensor requires a gradient, and autograd does not record this call; pass its "
                         "detach(), or call in torch.no_grad() or from an autograd.Function")


def _current() -> int:
    """The current device, and the dtype tables filled."""
    if not _matrix_types:
        _fill_types()
    return _current_device()


def _matrix(t, what: str, cur: int) -> Matrix:
    """The C struct of a 2-D device tensor whose rows are contiguous."""
    kind = _matrix_types.get(t.dtype)
    strides = t.stride()
    if kind is None or len(strides) != 2:
        raise ValueError(f"{what}: a 2-D tensor of one of {tuple(_LIST_TYPES)} expected, got {t.dtype} "
                         f"{tuple(t.shape)}")
    rows, cols = t.shape
    stride, inner = strides
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be neighbours")
    if t.get_device() != cur:
        _check_current(t, what, cur)
    if t.requires_grad:
        _refuse_grad(t, what)
    if rows <= 1 or not cols:  # the strides of a single row, or of no elements, have no meaning (torch may give any)
        stride = cols
    return Matrix(t.data_ptr(), rows, cols, stride, kind)


def _block8(codes, scales, what: str, cur: int, blocks: Optional[str] = None) -> Block8:
    """The C struct of a matrix in the 8-bit form.  The kind of its blocks
    follows from the scales' shape where it is not given (a single row has
    the same scales in both)."""
    strides, sstrides = codes.stride(), scales.stride()
    if codes.dtype not in _code_types or scales.dtype not in _scale_types or len(strides) != 2 or len(sstrides) != 2:
        raise ValueError(f"{what}: 2-D codes of {_CODES} and scales of {_SCALES} expected, got {codes.dtype} "
                         f"{tuple(codes.shape)} and {scales.dtype} {tuple(scales.shape)}")
    rows, cols = codes.shape
    srows, across = scales.shape
    by_rows = srows == rows if blocks is None else blocks == "rows"
    if across != (cols + 127) // 128 or srows != (rows if by_rows else (rows + 127) // 128):
        raise ValueError(f"{what}: scales of {(srows, across)} for codes of {(rows, cols)}, expected "
                         f"({rows} or {-(-rows // BLOCK8)}, {-(-cols // BLOCK8)}) by rows or tiles")
    stride, inner = strides
    sstride, sinner = sstrides
    if (inner != 1 and cols > 1) or (sinner != 1 and across > 1):
        raise ValueError(f"{what}: the bytes of a row must be neighbours")
    if codes.get_device() != cur or scales.get_device() != cur:
        _check_current(codes, what, cur)
        _check_current(scales, what, cur)
    if codes.requires_grad or scales.requires_grad:
        _refuse_grad(codes, what)
    # the strides of a single row, or of no elements, have no meaning (torch may give any)
    if rows <= 1 or not cols:
        stride = (cols + 15) & ~15
    if srows <= 1 or not cols:
        sstride = (across + 3) & ~3
    return Block8(codes.data_ptr(), scales.data_ptr(), rows, cols, stride, sstride, 0 if by_rows else 1)


def _blocks(name: str) -> str:
    if name not in BLOCKS:
        raise ValueError(f"blocks: {name!r}, expected one of {tuple(BLOCKS)}")
    return name


def _vector(t, n: int, what: str, cur: int, any_type: bool = False) -> int:
    """The address of a contiguous device vector of n float32 (any_type: or
    16-bit) elements."""
    if t.shape != (n,):
        raise ValueError(f"{what}: {n} elements expected, got a tensor of {tuple(t.shape)}")
    kind = _matrix_types.get(t.dtype)
    if kind is None or not (any_type or kind == TYPE_F32):
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {tuple(_LIST_TYPES) if any_type else 'float32'}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if t.get_device() != cur:
        _check_current(t, what, cur)
    if t.requires_grad:
        _refuse_grad(t, what)
    return t.data_ptr()


def _scratch(ws, need: int, what: str, cur: int) -> Optional[int]:
    """The address of a workspace of at least ``need`` bytes (None for 0)."""
    if need == 0:
        return None
    if ws is None or ws.numel() * ws.element_size() < need or not ws.is_contiguous():
        raise ValueError(f"{what}: a contiguous device tensor of at least {need} bytes")
    _check_current(ws, what, cur)
    return ws.data_ptr()


def _ref(x):
    return None if x is None else C.byref(x)


_increment_version = None


def _written(tensors):
    """Tells autograd that a call writes these tensors, as torch's in-place
    operations do: a backward pass that has saved one of them before raises."""
    global _increment_version
    if _increment_version is None:
        from torch.autograd.graph import increment_version
        _increment_version = increment_version
    _increment_version(tensors)


def block8_buffers(rows: int, cols: int, blocks: str = "rows", device=None):
    """New (codes, scales) tensors for a matrix of rows x cols in the 8-bit
    form, filled with zeros: views [rows, cols] and [rows or tiles of 128 rows,
    blocks of 128 columns] of buffers whose rows are padded to 16 and 4 bytes,
    as the calls want them."""
    import torch
    if rows < 0 or cols < 0:
        raise ValueError(f"block8_buffers: {rows} x {cols}")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    across = -(-cols // BLOCK8)
    srows = rows if _blocks(blocks) == "rows" else -(-rows // BLOCK8)
    codes = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=device)
    scales = torch.zeros(srows, -(-across // 4) * 4, dtype=torch.uint8, device=device)
    return (codes.view(torch.float8_e4m3fn)[:, :cols], scales.view(torch.float8_e8m0fnu)[:, :across])


def block8_encode(x, codes=None, scales=None, codes_t=None, scales_t=None, blocks: str = "rows", row_mul=None,
                  col_mul=None, stream=None):
    """A float32, float16 or bfloat16 matrix, or x * row_mul[:, None] * col_mul,
    into the 8-bit form: ``codes`` and ``scales`` as it is, ``codes_t`` and
    ``scales_t`` transposed (either pair may be None).  ``blocks``: "rows" (128
    values along a row of the codes share a scale) or "tiles" (128 x 128).

    Autograd does not record this call or the norm and product below: where it
    would have to (grad mode on, a tensor that requires a gradient) they raise
    ValueError."""
    cur = _current()
    _blocks(blocks)
    mx = _matrix(x, "matrix", cur)
    if (codes is None) != (scales is None) or (codes_t is None) != (scales_t is None):
        raise ValueError("codes and scales come together")
    out = None if codes is None else _block8(codes, scales, "codes", cur, blocks)
    out_t = None if codes_t is None else _block8(codes_t, scales_t, "transposed codes", cur, blocks)
    rm = None if row_mul is None else _vector(row_mul, mx.rows, "row multipliers", cur)
    cm, ctype = None, TYPE_NONE
    if col_mul is not None:
        cm = _vector(col_mul, mx.cols, "column multipliers", cur, True)
        ctype = _matrix_types[col_mul.dtype]
    _check(lib().zero_block8_encode(C.byref(mx), rm, cm, ctype, _ref(out), _ref(out_t), _stream_on(cur, stream)),
           "zero_block8_encode")
    _written([t for t in (codes, scales, codes_t, scales_t) if t is not None])


def rms_norm8(x, weight, codes, scales, rstd, residual=None, h=None, eps: float = 1e-6, stream=None):
    """The root-mean-square norm of x (+ residual) times ``weight``, in the 8-bit
    form by rows.  ``rstd`` (float32 [rows]) and with a residual ``h`` (the sum, of
    x's dtype; may be x or residual itself) are written for the backward pass."""
    cur = _current()
    mx = _matrix(x, "x", cur)
    mr = None if residual is None else _matrix(residual, "residual", cur)
    mh = None if h is None else _matrix(h, "h", cur)
    w = _vector(weight, mx.cols, "weight", cur, True)
    r = _vector(rstd, mx.rows, "rstd", cur)
    _check(lib().zero_rms_norm8(C.byref(mx), _ref(mr), w, _matrix_types[weight.dtype], float(eps), _ref(mh),
                                C.byref(_block8(codes, scales, "codes", cur, "rows")), r, _stream_on(cur, stream)),
           "zero_rms_norm8")
    _written((codes, scales, rstd) if h is None else (codes, scales, rstd, h))


def rms_norm8_workspace_bytes(rows: int, cols: int) -> int:
    return lib().zero_rms_norm8_workspace_bytes(rows, cols)


def rms_norm8_backward(dy, h, weight, rstd, dx, dweight=None, workspace=None, dh=None, stream=None):
    """rms_norm8's gradients: ``dx`` (of x and of residual; may be dy or dh
    itself) and ``dweight`` (float32, or None).  ``h``: rms_norm8's h, or its x
    where it had no residual.  ``dh``: what reaches h another way.  ``workspace``:
    of rms_norm8_workspace_bytes() bytes, for dweight, not shared with a call
    that may run at the same time."""
    cur = _current()
    my, mh, mx = _matrix(dy, "dy", cur), _matrix(h, "h", cur), _matrix(dx, "dx", cur)
    md = None if dh is None else _matrix(dh, "dh", cur)
    w = _vector(weight, my.cols, "weight", cur, True)
    r = _vector(rstd, my.rows, "rstd", cur)
    dw = ws = None
    if dweight is not None:
        dw = _vector(dweight, my.cols, "dweight", cur)
        ws = _scratch(workspace, rms_norm8_workspace_bytes(my.rows, my.cols), "workspace", cur)
    _check(lib().zero_rms_norm8_backward(C.byref(my), C.byref(mh), w, _matrix_types[weight.dtype], r, _ref(md),
                                         C.byref(mx), dw, ws, _stream_on(cur, stream)), "zero_rms_norm8_backward")
    _written(dx if dweight is None else (dx, dweight))


def block8_workspace_bytes(m: int, n: int, k: int) -> int:
    return lib().zero_block8_workspace_bytes(m, n, k)


def block8_product(a, a_scales, b, b_scales, out, add=None, workspace=None, stream=None):
    """out = a b^T (+ add) of two matrices in the 8-bit form, [M, K] and [N, K].
    ``add``: of out's dtype and shape; may be out itself.  ``workspace``: of
    block8_workspace_bytes(M, N, K) bytes (may be None if that is 0), not shared
    with a call that may run at the same time.  ``out`` in float32: sums in
    float32; in 16 bits: twice as fast, on instructions that add eight
    neighbouring k in fewer bits (include/zero_dp.h states the bound)."""
    cur = _current()
    ma, mb = _block8(a, a_scales, "a", cur), _block8(b, b_scales, "b", cur)
    mo = _matrix(out, "out", cur)
    mc = None if add is None else _matrix(add, "add", cur)
    ws = _scratch(workspace, block8_workspace_bytes(ma.rows, mb.rows, ma.cols), "workspace", cur)
    _check(lib().zero_block8_product(C.byref(ma), C.byref(mb), _ref(mc), C.byref(mo), ws, _stream_on(cur, stream)),
           "zero_block8_product")
    _written(out)


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
