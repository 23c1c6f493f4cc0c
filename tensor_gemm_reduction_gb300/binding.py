"""Python binding of the C ABI in ``include/gsr.h``: argument marshalling only.

Every function here has the name of the C entry point it calls. Tensors are
checked for dtype, device, contiguity and shape, turned into raw pointers and
passed to the library with the current CUDA stream; all arithmetic runs in the
library's kernels. There is no fallback: if the library has not been built, the
first call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libgsr.so")
_lib = None

GSR_OK = 0
GSR_ERR_INVALID_VALUE = 1
GSR_ERR_UNSUPPORTED = 2
GSR_ERR_WORKSPACE = 3
GSR_ERR_CUDA = 4
GSR_ERR_TIMEOUT = 5
GSR_MAX_SHARDS = 16

GSR_OPT_SPLIT_K = 1
GSR_OPT_BLOCK_N = 2
GSR_OPT_TIMEOUT_NS = 3
GSR_OPT_MAX_CTAS = 4
GSR_OPT_RASTER_M = 5
GSR_OPT_L2_HINTS = 6
GSR_OPT_CTA_GROUP = 7
GSR_OPT_SCHEDULE = 8
GSR_OPT_SMALL_M = 9
GSR_OPT_SMALL_TILE_ROWS = 10
GSR_OPT_RASTER_N = 11
GSR_OPT_SMALL_KBLOCKS = 12

MODE_AR, MODE_RS, MODE_AG = 0, 1, 2

_STATUS_NAMES = {
    GSR_OK: "GSR_OK",
    GSR_ERR_INVALID_VALUE: "GSR_ERR_INVALID_VALUE",
    GSR_ERR_UNSUPPORTED: "GSR_ERR_UNSUPPORTED",
    GSR_ERR_WORKSPACE: "GSR_ERR_WORKSPACE",
    GSR_ERR_CUDA: "GSR_ERR_CUDA",
    GSR_ERR_TIMEOUT: "GSR_ERR_TIMEOUT",
}

EXPORTED = (
    "gemm_shard_plan_create", "gemm_shard_plan_create_host", "gemm_shard_plan_destroy", "gemm_shard_plan_set_option",
    "gemm_shard_workspace_size", "gemm_shard_workspace_init", "gemm_ar", "gemm_rs",
    "gemm_ag", "gemm_shard_check_status", "gsr_last_error_string", "gemm_shard_describe",
    "gemm_ar_noalloc", "gemm_ag_flagged", "gemm_shard_signal", "gemm_ar_replicated",
    "gemm_shard_pack_gather", "gemm_ar_noalloc_check_status",
    "gemm_routed_workspace_size", "gemm_routed_workspace_init", "gemm_group_route",
    "gemm_grouped", "gemm_grouped_gated", "gemm_group_combine", "gemm_ar_lora",
    "gemm_shard_rms_norm", "gemm_shard_quantize", "gemm_ar_fp8", "gemm_ag_fp8",
    "gemm_expert_layer",
)


class GsrConfig(ctypes.Structure):
    """Mirror of gsr_config (include/gsr.h)."""
    _fields_ = [("block_n", ctypes.c_int), ("cta_group", ctypes.c_int),
                ("schedule", ctypes.c_int), ("split", ctypes.c_int),
                ("tiles", ctypes.c_int64), ("dp_tiles", ctypes.c_int64),
                ("sk_iters", ctypes.c_int64), ("ctas", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t), ("kblocks", ctypes.c_int),
                ("l2_hints", ctypes.c_int)]


class GsrError(RuntimeError):
    """A non-zero gsr_status, with the library's message."""

    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load the built library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"the CUDA library {_LIB_PATH} is not built; run "
            "`python -m tensor_gemm_reduction_gb300.build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    ptr_arr = ctypes.POINTER(ctypes.c_void_p)
    i64_arr = ctypes.POINTER(ctypes.c_int64)
    lib.gemm_shard_plan_create.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i64, i32]
    lib.gemm_shard_plan_create_host.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i64, i32]
    lib.gemm_shard_plan_destroy.argtypes = [vp]
    lib.gemm_shard_plan_set_option.argtypes = [vp, i32, i64]
    lib.gemm_shard_workspace_size.argtypes = [vp]
    lib.gemm_shard_workspace_size.restype = sz
    lib.gemm_shard_workspace_init.argtypes = [vp, vp, sz, vp]
    lib.gemm_ar.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, vp, vp, sz, vp]
    lib.gemm_rs.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, ptr_arr, vp, sz, vp]
    lib.gemm_ar_replicated.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, ptr_arr, vp,
                                       sz, vp]
    lib.gemm_ag.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, vp, vp, vp, sz, vp]
    lib.gemm_ar_noalloc.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, vp, vp]
    lib.gemm_ag_flagged.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, vp, vp, vp,
                                    ctypes.c_uint32, vp, sz, vp]
    lib.gemm_shard_signal.argtypes = [vp, vp, ctypes.c_uint32, vp]
    lib.gemm_shard_pack_gather.argtypes = [vp, i32, i64_arr, i32, i64, ptr_arr, i64, vp, vp, sz, vp]
    lib.gemm_shard_check_status.argtypes = [vp, vp, vp]
    lib.gemm_ar_noalloc_check_status.argtypes = [vp, vp]
    lib.gemm_routed_workspace_size.argtypes = [vp]
    lib.gemm_routed_workspace_size.restype = sz
    lib.gemm_routed_workspace_init.argtypes = [vp, vp, sz, vp]
    lib.gemm_group_route.argtypes = [vp, i64, i32, i32, vp, i32, vp, vp, vp, vp]
    lib.gemm_grouped.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.gemm_grouped_gated.argtypes = lib.gemm_grouped.argtypes
    lib.gemm_group_combine.argtypes = [vp, i64, i32, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.gemm_ar_lora.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, i32, i32, ptr_arr,
                                 vp, vp, vp, vp, vp, sz, vp]
    lib.gemm_shard_rms_norm.argtypes = [vp, i64, i64, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp]
    lib.gemm_shard_quantize.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp]
    lib.gemm_ar_fp8.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, ptr_arr, ptr_arr, vp,
                                vp, sz, vp]
    lib.gemm_ag_fp8.argtypes = [vp, i64, i64, i32, i64_arr, ptr_arr, ptr_arr, vp, vp, vp, vp, sz, vp]
    lib.gemm_expert_layer.argtypes = [vp, i64, i32, i32, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gsr_last_error_string.restype = ctypes.c_char_p
    lib.gemm_shard_describe.argtypes = [vp, i32, i64, i64, i64, i32, i64_arr,
                                        ctypes.POINTER(GsrConfig)]
    for name in EXPORTED:
        if name not in ("gemm_shard_workspace_size", "gemm_routed_workspace_size",
                        "gsr_last_error_string"):
            getattr(lib, name).restype = i32
    _lib = lib
    return lib


def gsr_last_error_string() -> str:
    return load_library().gsr_last_error_string().decode()


def _check(status: int) -> None:
    if status != GSR_OK:
        raise GsrError(status, gsr_last_error_string())


class Plan:
    """Owns a gemm_shard_plan handle; destroyed with the object."""

    def __init__(self, handle: int, device: int, max_M: int, max_N: int, max_K: int, max_R: int):
        self.handle = ctypes.c_void_p(handle)
        self.device, self.max_M, self.max_N, self.max_K, self.max_R = device, max_M, max_N, max_K, max_R

    def __del__(self):
        if getattr(self, "handle", None) and self.handle.value and _lib is not None:
            _lib.gemm_shard_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p(0)


def gemm_shard_plan_create(device: int, max_M: int, max_N: int, max_K: int, max_R: int) -> Plan:
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.gemm_shard_plan_create(ctypes.byref(h), int(device), int(max_M), int(max_N),
                                      int(max_K), int(max_R)))
    return Plan(h.value, device, max_M, max_N, max_K, max_R)


def gemm_shard_plan_create_host(sm_count: int, max_M: int, max_N: int, max_K: int,
                                max_R: int) -> Plan:
    """A plan bound to no device (argument checks, configuration, workspace size)."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.gemm_shard_plan_create_host(ctypes.byref(h), int(sm_count), int(max_M),
                                           int(max_N), int(max_K), int(max_R)))
    return Plan(h.value, -1, max_M, max_N, max_K, max_R)


def gemm_shard_plan_destroy(plan: Plan) -> None:
    if plan.handle.value:
        _check(load_library().gemm_shard_plan_destroy(plan.handle))
        plan.handle = ctypes.c_void_p(0)


def gemm_shard_plan_set_option(plan: Plan, option: int, value: int) -> None:
    _check(load_library().gemm_shard_plan_set_option(plan.handle, int(option), int(value)))


def gemm_shard_workspace_size(plan: Plan) -> int:
    return int(load_library().gemm_shard_workspace_size(plan.handle))


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        # The raw handle: building a torch.cuda.Stream took 3 us, as long as a launch.
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def _ws(ws: torch.Tensor):
    if not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def gemm_shard_workspace_alloc(plan: Plan) -> torch.Tensor:
    """A workspace tensor of gemm_shard_workspace_size bytes (torch allocates it)."""
    n = gemm_shard_workspace_size(plan)
    return torch.empty(n, dtype=torch.uint8, device=f"cuda:{plan.device}")


def gemm_shard_workspace_init(plan: Plan, ws: torch.Tensor, stream=None) -> None:
    p, n = _ws(ws)
    _check(load_library().gemm_shard_workspace_init(plan.handle, p, n, _stream(stream)))


_BF16 = torch.bfloat16


def _bf16_2d(t: torch.Tensor, name: str) -> None:
    if t.dtype is not _BF16 or not t.is_cuda or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D bf16 CUDA tensor")


class PreparedCall:
    """A validated, marshalled call of one entry point on fixed buffers.

    Serving loops reuse the same shard, output and workspace buffers every
    step; preparing the call once moves the per-call Python cost to a single
    ctypes call. The buffers must stay alive and keep their shapes; their
    contents may change. The stream is read at each call unless fixed."""

    def __init__(self, fn, args, keep, stream=None):
        self._fn, self._args, self._keep = fn, args, keep
        self._stream = None if stream is None else _stream(stream)

    def __call__(self, stream=None):
        st = self._stream if stream is None and self._stream is not None else _stream(stream)
        _check(self._fn(*self._args, st))


def _ptrs(ts: Sequence[Optional[torch.Tensor]]):
    arr = (ctypes.c_void_p * len(ts))(*[t.data_ptr() if t is not None else 0 for t in ts])
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), arr


def _i64s(vals: Sequence[int]):
    arr = (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])
    return ctypes.cast(arr, ctypes.POINTER(ctypes.c_int64)), arr


def _ar_args(plan, X_r, W_r, Y, ws):
    R = len(X_r)
    if R != len(W_r) or R == 0:
        raise ValueError("X_r and W_r need the same, non-zero number of shards")
    _bf16_2d(Y, "Y")
    M, N = Y.shape
    K_r = []
    for r in range(R):
        x, w = X_r[r], W_r[r]
        _bf16_2d(x, f"X_r[{r}]")
        _bf16_2d(w, f"W_r[{r}]")
        k = x.shape[1]
        if x.shape[0] != M or w.shape[0] != N or w.shape[1] != k:
            raise ValueError(f"shard {r}: X_r must be {M} x K_r and W_r {N} x K_r")
        K_r.append(k)
    k, ka = _i64s(K_r)
    xp, xa = _ptrs(X_r)
    wp, wa = _ptrs(W_r)
    wsp, wsn = _ws(ws)
    args = (plan.handle, M, N, R, k, xp, wp, ctypes.c_void_p(Y.data_ptr()), wsp, wsn)
    return args, (ka, xa, wa, X_r, W_r, Y, ws)


def gemm_ar(plan: Plan, X_r: Sequence[torch.Tensor], W_r: Sequence[torch.Tensor],
            Y: torch.Tensor, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = sum_r X_r @ W_r.T (X_r: M x K_r, W_r: N x K_r, Y: M x N, all bf16)."""
    args, keep = _ar_args(plan, X_r, W_r, Y, ws)
    _check(load_library().gemm_ar(*args, _stream(stream)))
    return Y


def prepare_ar(plan: Plan, X_r, W_r, Y, ws, stream=None) -> PreparedCall:
    """gemm_ar on fixed buffers, validated and marshalled once."""
    args, keep = _ar_args(plan, X_r, W_r, Y, ws)
    return PreparedCall(load_library().gemm_ar, args, keep, stream)


def gemm_ar_replicated(plan: Plan, X_r: Sequence[torch.Tensor], W_r: Sequence[torch.Tensor],
                       Y_r: Sequence[torch.Tensor], ws: torch.Tensor, stream=None):
    """Y_r[r] = sum_q X_q @ W_q.T for every r (R outputs of M x N, all bf16)."""
    R = len(X_r)
    if len(Y_r) != R:
        raise ValueError("need one output per shard")
    for r in range(R):
        _bf16_2d(Y_r[r], f"Y_r[{r}]")
        if Y_r[r].shape != Y_r[0].shape:
            raise ValueError("all outputs must have the same shape")
    args, keep = _ar_args(plan, X_r, W_r, Y_r[0], ws)
    yp, ya = _ptrs(Y_r)
    # same marshalling as gemm_ar, with the output pointer array in place of Y
    args = args[:7] + (yp,) + args[8:]
    _check(load_library().gemm_ar_replicated(*args, _stream(stream)))
    return Y_r


def gemm_ar_noalloc(plan: Plan, X_r: Sequence[torch.Tensor], W_r: Sequence[torch.Tensor],
                    Y: torch.Tensor, stream=None) -> torch.Tensor:
    """gemm_ar for callers that cannot allocate device memory: no workspace; the
    library's built-in 24 MiB device scratch is used (shared by every call on a
    device, so calls must not overlap on the GPU)."""
    R = len(X_r)
    if R != len(W_r) or R == 0:
        raise ValueError("X_r and W_r need the same, non-zero number of shards")
    for r in range(R):
        _bf16_2d(X_r[r], f"X_r[{r}]")
        _bf16_2d(W_r[r], f"W_r[{r}]")
    _bf16_2d(Y, "Y")
    M, N = Y.shape
    K_r = [x.shape[1] for x in X_r]
    for r in range(R):
        if X_r[r].shape[0] != M or W_r[r].shape != (N, K_r[r]):
            raise ValueError(f"shard {r}: X_r must be {M} x K_r and W_r {N} x K_r")
    k, ka = _i64s(K_r)
    xp, xa = _ptrs(X_r)
    wp, wa = _ptrs(W_r)
    _check(load_library().gemm_ar_noalloc(plan.handle, M, N, R, k, xp, wp,
                                          ctypes.c_void_p(Y.data_ptr()), _stream(stream)))
    return Y


def gemm_ar_noalloc_check_status(plan: Plan, stream=None) -> None:
    """Synchronise, then raise GsrError(GSR_ERR_TIMEOUT) if the last
    gemm_ar_noalloc call on the plan's device had an in-kernel wait run out."""
    _check(load_library().gemm_ar_noalloc_check_status(plan.handle, _stream(stream)))


def _rs_args(plan, X_r, W_r, Y_r, ws, M=None):
    R = len(X_r)
    if R != len(W_r) or R != len(Y_r) or R == 0:
        raise ValueError("X_r, W_r and Y_r need the same, non-zero number of shards")
    M = X_r[0].shape[0] if M is None else int(M)
    N = W_r[0].shape[0]
    rps = -(-M // R)
    K_r = []
    for r in range(R):
        _bf16_2d(X_r[r], f"X_r[{r}]")
        _bf16_2d(W_r[r], f"W_r[{r}]")
        _bf16_2d(Y_r[r], f"Y_r[{r}]")
        k = X_r[r].shape[1]
        if X_r[r].shape[0] != M or W_r[r].shape != (N, k):
            raise ValueError(f"shard {r}: X_r must be {M} x K_r and W_r {N} x K_r")
        if Y_r[r].shape[0] < rps or Y_r[r].shape[1] != N:
            raise ValueError(f"Y_r[{r}] must hold at least {rps} rows of {N}")
        K_r.append(k)
    k, ka = _i64s(K_r)
    xp, xa = _ptrs(X_r)
    wp, wa = _ptrs(W_r)
    yp, ya = _ptrs(Y_r)
    wsp, wsn = _ws(ws)
    args = (plan.handle, M, N, R, k, xp, wp, yp, wsp, wsn)
    return args, (ka, xa, wa, ya, X_r, W_r, Y_r, ws)


def gemm_rs(plan: Plan, X_r: Sequence[torch.Tensor], W_r: Sequence[torch.Tensor],
            Y_r: Sequence[torch.Tensor], ws: torch.Tensor, M: Optional[int] = None,
            stream=None) -> Sequence[torch.Tensor]:
    """Y_r[s] = rows [s*rps, min(M,(s+1)*rps)) of sum_r X_r @ W_r.T, rps = ceil(M/R)."""
    args, keep = _rs_args(plan, X_r, W_r, Y_r, ws, M)
    _check(load_library().gemm_rs(*args, _stream(stream)))
    return Y_r


def prepare_rs(plan: Plan, X_r, W_r, Y_r, ws, M=None, stream=None) -> PreparedCall:
    """gemm_rs on fixed buffers, validated and marshalled once."""
    args, keep = _rs_args(plan, X_r, W_r, Y_r, ws, M)
    return PreparedCall(load_library().gemm_rs, args, keep, stream)


def _ag_call_args(plan, A_r, W, Y, ws):
    N, K, M_r = _ag_args(A_r, W, Y)
    m, ma = _i64s(M_r)
    ap, aa = _ptrs([a if a.numel() else None for a in A_r])
    wsp, wsn = _ws(ws)
    args = (plan.handle, N, K, len(A_r), m, ap, ctypes.c_void_p(W.data_ptr()),
            ctypes.c_void_p(Y.data_ptr()), wsp, wsn)
    return args, (ma, aa, A_r, W, Y, ws)


def gemm_ag(plan: Plan, A_r: Sequence[torch.Tensor], W: torch.Tensor, Y: torch.Tensor,
            ws: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = cat(A_r) @ W.T (A_r: M_r x K, W: N x K, Y: sum(M_r) x N, all bf16)."""
    args, keep = _ag_call_args(plan, A_r, W, Y, ws)
    _check(load_library().gemm_ag(*args, _stream(stream)))
    return Y


def prepare_ag(plan: Plan, A_r, W, Y, ws, stream=None) -> PreparedCall:
    """gemm_ag on fixed buffers, validated and marshalled once."""
    args, keep = _ag_call_args(plan, A_r, W, Y, ws)
    return PreparedCall(load_library().gemm_ag, args, keep, stream)


def _ag_args(A_r, W, Y):
    R = len(A_r)
    if R == 0:
        raise ValueError("need at least one shard")
    _bf16_2d(W, "W")
    _bf16_2d(Y, "Y")
    N, K = W.shape
    M_r = []
    for r, a in enumerate(A_r):
        if a.numel() == 0:
            M_r.append(0)
            continue
        _bf16_2d(a, f"A_r[{r}]")
        if a.shape[1] != K:
            raise ValueError(f"A_r[{r}] must have K={K} columns")
        M_r.append(a.shape[0])
    if Y.shape != (sum(M_r), N):
        raise ValueError(f"Y must be {sum(M_r)} x {N}")
    return N, K, M_r


def gemm_ag_flagged(plan: Plan, A_r: Sequence[torch.Tensor], W: torch.Tensor, Y: torch.Tensor,
                    ready: torch.Tensor, epoch: int, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """gemm_ag that waits in the kernel until ready[r] reaches epoch before reading A_r.
    `ready` is a CUDA int32/uint32 tensor of R words."""
    N, K, M_r = _ag_args(A_r, W, Y)
    if not ready.is_cuda or ready.numel() < len(A_r) or ready.element_size() != 4:
        raise ValueError("ready must be a CUDA tensor of R 32-bit words")
    m, ma = _i64s(M_r)
    ap, aa = _ptrs([a if a.numel() else None for a in A_r])
    wsp, wsn = _ws(ws)
    _check(load_library().gemm_ag_flagged(plan.handle, N, K, len(A_r), m, ap,
                                          ctypes.c_void_p(W.data_ptr()),
                                          ctypes.c_void_p(Y.data_ptr()),
                                          ctypes.c_void_p(ready.data_ptr()),
                                          ctypes.c_uint32(epoch & 0xFFFFFFFF), wsp, wsn,
                                          _stream(stream)))
    return Y


def gemm_shard_signal(plan: Plan, flag_ptr: int, value: int, stream=None) -> None:
    """Enqueue a write of `value` to the device word at `flag_ptr` on `stream`."""
    _check(load_library().gemm_shard_signal(plan.handle, ctypes.c_void_p(int(flag_ptr)),
                                            ctypes.c_uint32(value & 0xFFFFFFFF), _stream(stream)))


def gemm_shard_check_status(plan: Plan, ws: torch.Tensor, stream=None) -> None:
    p, _ = _ws(ws)
    _check(load_library().gemm_shard_check_status(plan.handle, p, _stream(stream)))


def gemm_shard_describe(plan: Plan, mode: int, M: int, N: int, K: int,
                        sizes: Sequence[int]) -> dict:
    lib = load_library()
    s, sa = _i64s(sizes)
    cfg = GsrConfig()
    _check(lib.gemm_shard_describe(plan.handle, int(mode), int(M), int(N), int(K), len(sizes), s,
                                   ctypes.byref(cfg)))
    return {name: getattr(cfg, name) for name, _ in GsrConfig._fields_}


def _pack_args(plan, S, rows_out, P, ws):
    R = len(S)
    if R == 0 or any(len(s) != len(S[0]) for s in S) or not S[0]:
        raise ValueError("S must hold R >= 1 shards with the same T >= 1 states each")
    T = len(S[0])
    _bf16_2d(P, "P")
    H = P.shape[1] // T
    if P.shape != (rows_out, T * H) or H * T != P.shape[1]:
        raise ValueError(f"P must be rows_out x (T*H) = {rows_out} x {T}*H")
    M_r, flat = [], []
    for r, states in enumerate(S):
        m = states[0].shape[0]
        for t, st in enumerate(states):
            if st.numel() == 0 and m == 0:
                flat.append(None)
                continue
            _bf16_2d(st, f"S[{r}][{t}]")
            if st.shape != (m, H):
                raise ValueError(f"S[{r}][{t}] must be {m} x {H}")
            flat.append(st)
        M_r.append(m)
    m, ma = _i64s(M_r)
    sp, sa = _ptrs(flat)
    wsp, wsn = _ws(ws)
    args = (plan.handle, R, m, T, H, sp, rows_out, ctypes.c_void_p(P.data_ptr()), wsp, wsn)
    return args, (ma, sa, S, P, ws)


def gemm_shard_pack_gather(plan: Plan, S: Sequence[Sequence[torch.Tensor]], rows_out: int,
                           P: torch.Tensor, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """P[g, t*H:(t+1)*H] = cat_r(S[r][t])[g] for g < rows_out (S[r][t]: M_r x H, bf16;
    P: rows_out x T*H). Returns P; the state-t view is P[:, t*H:(t+1)*H]."""
    args, keep = _pack_args(plan, S, rows_out, P, ws)
    _check(load_library().gemm_shard_pack_gather(*args, _stream(stream)))
    return P


def prepare_pack_gather(plan: Plan, S, rows_out, P, ws, stream=None) -> PreparedCall:
    """gemm_shard_pack_gather on fixed buffers, validated and marshalled once."""
    args, keep = _pack_args(plan, S, rows_out, P, ws)
    return PreparedCall(load_library().gemm_shard_pack_gather, args, keep, stream)


# ------------------------------------------------------------ routed projections

def gemm_routed_workspace_size(plan: Plan) -> int:
    return int(load_library().gemm_routed_workspace_size(plan.handle))


def gemm_routed_workspace_alloc(plan: Plan) -> torch.Tensor:
    """A workspace tensor of gemm_routed_workspace_size bytes (torch allocates it)."""
    n = gemm_routed_workspace_size(plan)
    return torch.empty(n, dtype=torch.uint8, device=f"cuda:{plan.device}")


def gemm_routed_workspace_init(plan: Plan, ws: torch.Tensor, stream=None) -> None:
    p, n = _ws(ws)
    _check(load_library().gemm_routed_workspace_init(plan.handle, p, n, _stream(stream)))


def _dense(t: torch.Tensor, name: str, dtype, shape=None, dim=None) -> None:
    """A contiguous CUDA tensor of the dtype and, where given, shape (None: any size)."""
    dim = dim if shape is None else len(shape)
    ok = t.dtype is dtype and t.is_cuda and t.dim() == dim and t.is_contiguous()
    if ok and shape is not None:
        ok = all(want is None or want == have for want, have in zip(shape, t.shape))
    if not ok:
        size = f"{dim}-D" if shape is None else "x".join("?" if s is None else str(s) for s in shape)
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of {size}, "
                         f"not {t.dtype} {tuple(t.shape)}")


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None and t.numel() else 0)


def _route_args(plan, ids, E, offsets, source, position):
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be int32 or int64")
    _dense(ids, "ids", ids.dtype, dim=2)
    T, topk = ids.shape
    _dense(offsets, "offsets", torch.int32, (int(E) + 1,))
    _dense(source, "source", torch.int32, (T * topk,))
    _dense(position, "position", torch.int32, (T, topk))
    args = (plan.handle, T, topk, int(E), _ptr(ids), ids.element_size(), _ptr(offsets),
            _ptr(source), _ptr(position))
    return args, (ids, offsets, source, position)


def gemm_group_route(plan: Plan, ids: torch.Tensor, E: int, offsets: torch.Tensor,
                     source: torch.Tensor, position: torch.Tensor, stream=None):
    """Group the entries of ids (T x topk, int32 or int64; outside 0..E-1: dropped) by expert.

    Writes offsets (E + 1), source (T * topk: the token of each sorted row, -1
    past the kept ones) and position (T x topk: the sorted row of each entry, -1
    if dropped), all int32, and returns them."""
    args, _ = _route_args(plan, ids, E, offsets, source, position)
    _check(load_library().gemm_group_route(*args, _stream(stream)))
    return offsets, source, position


def prepare_group_route(plan: Plan, ids, E, offsets, source, position, stream=None) -> PreparedCall:
    """gemm_group_route on fixed buffers, validated and marshalled once."""
    args, keep = _route_args(plan, ids, E, offsets, source, position)
    return PreparedCall(load_library().gemm_group_route, args, keep, stream)


def _grouped_args(plan, X, W, offsets, Y, ws, rows, gated):
    _bf16_2d(X, "X")
    _dense(W, "W", _BF16, dim=3)
    E, wide, K = W.shape
    if gated and wide % 2:
        raise ValueError("W must hold as many gate as up rows")
    N = wide // 2 if gated else wide
    _dense(Y, "Y", _BF16, (None, N))
    M = Y.shape[0]
    _dense(offsets, "offsets", torch.int32, (E + 1,))
    if X.shape[1] != K or (rows is None and X.shape[0] < M):
        raise ValueError(f"X must have K={K} columns" + ("" if rows is not None else f" and at least {M} rows"))
    if rows is not None:
        _dense(rows, "rows", torch.int32, (M,))
    wsp, wsn = _ws(ws)
    args = (plan.handle, E, M, N, K, _ptr(offsets), X.shape[0], _ptr(X), _ptr(rows), _ptr(W), _ptr(Y),
            wsp, wsn)
    return args, (X, W, offsets, Y, ws, rows)


def gemm_grouped(plan: Plan, X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor,
                 Y: torch.Tensor, ws: torch.Tensor, rows: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Y[i] = X[i] @ W[e].T for offsets[e] <= i < offsets[e+1] (W: E x N x K); with
    `rows`, X[rows[i]] in place of X[i]. Rows of no group are not written."""
    args, _ = _grouped_args(plan, X, W, offsets, Y, ws, rows, False)
    _check(load_library().gemm_grouped(*args, _stream(stream)))
    return Y


def prepare_grouped(plan: Plan, X, W, offsets, Y, ws, rows=None, stream=None) -> PreparedCall:
    """gemm_grouped on fixed buffers, validated and marshalled once."""
    args, keep = _grouped_args(plan, X, W, offsets, Y, ws, rows, False)
    return PreparedCall(load_library().gemm_grouped, args, keep, stream)


def gemm_grouped_gated(plan: Plan, X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor,
                       Y: torch.Tensor, ws: torch.Tensor, rows: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Y[i] = silu(X[i] @ W[e, :N].T) * (X[i] @ W[e, N:].T) (W: E x 2N x K); otherwise
    as gemm_grouped."""
    args, _ = _grouped_args(plan, X, W, offsets, Y, ws, rows, True)
    _check(load_library().gemm_grouped_gated(*args, _stream(stream)))
    return Y


def prepare_grouped_gated(plan: Plan, X, W, offsets, Y, ws, rows=None, stream=None) -> PreparedCall:
    """gemm_grouped_gated on fixed buffers, validated and marshalled once."""
    args, keep = _grouped_args(plan, X, W, offsets, Y, ws, rows, True)
    return PreparedCall(load_library().gemm_grouped_gated, args, keep, stream)


def _combine_args(plan, Z, position, weights, Y, base):
    _bf16_2d(Z, "Z")
    _dense(position, "position", torch.int32, dim=2)
    T, topk = position.shape
    _dense(weights, "weights", torch.float32, (T, topk))
    _dense(Y, "Y", _BF16, (T, Z.shape[1]))
    if base is not None:
        _dense(base, "base", _BF16, (T, Z.shape[1]))
    args = (plan.handle, T, topk, Z.shape[1], Z.shape[0], _ptr(Z), _ptr(position), _ptr(weights),
            _ptr(base), _ptr(Y))
    return args, (Z, position, weights, Y, base)


def gemm_group_combine(plan: Plan, Z: torch.Tensor, position: torch.Tensor, weights: torch.Tensor,
                       Y: torch.Tensor, base: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[t] = base[t] + sum_j weights[t, j] * Z[position[t, j]] (position and weights:
    T x topk, int32 and fp32; a position outside Z adds nothing)."""
    args, _ = _combine_args(plan, Z, position, weights, Y, base)
    _check(load_library().gemm_group_combine(*args, _stream(stream)))
    return Y


def prepare_group_combine(plan: Plan, Z, position, weights, Y, base=None, stream=None) -> PreparedCall:
    """gemm_group_combine on fixed buffers, validated and marshalled once."""
    args, keep = _combine_args(plan, Z, position, weights, Y, base)
    return PreparedCall(load_library().gemm_group_combine, args, keep, stream)


def _layer_args(plan, X, ids, weights, W_up, W_down, Y, ws, base):
    _bf16_2d(X, "X")
    T, K = X.shape
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be int32 or int64")
    _dense(ids, "ids", ids.dtype, (T, None))
    topk = ids.shape[1]
    _dense(weights, "weights", torch.float32, (T, topk))
    _dense(W_up, "W_up", _BF16, (None, None, K))
    E, wide, _ = W_up.shape
    if wide % 2:
        raise ValueError("W_up must hold as many gate as up rows")
    N = wide // 2
    _dense(W_down, "W_down", _BF16, (E, K, N))
    _dense(Y, "Y", _BF16, (T, K))
    if base is not None:
        _dense(base, "base", _BF16, (T, K))
    wsp, wsn = _ws(ws)
    args = (plan.handle, T, topk, E, N, K, _ptr(ids), ids.element_size(), _ptr(weights), _ptr(X), _ptr(W_up),
            _ptr(W_down), _ptr(base), _ptr(Y), wsp, wsn)
    return args, (X, ids, weights, W_up, W_down, Y, ws, base)


def gemm_expert_layer(plan: Plan, X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, W_up: torch.Tensor,
                      W_down: torch.Tensor, Y: torch.Tensor, ws: torch.Tensor,
                      base: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[t] = base[t] + sum_j weights[t, j] * W_down[e] @ (silu(W_up[e, :N] @ X[t]) * (W_up[e, N:] @
    X[t])), e = ids[t, j] (int32 or int64; outside 0..E-1: dropped), for up to 64 tokens (W_up:
    E x 2N x K, W_down: E x K x N, weights: fp32; the routed workspace)."""
    args, _ = _layer_args(plan, X, ids, weights, W_up, W_down, Y, ws, base)
    _check(load_library().gemm_expert_layer(*args, _stream(stream)))
    return Y


def prepare_expert_layer(plan: Plan, X, ids, weights, W_up, W_down, Y, ws, base=None, stream=None) -> PreparedCall:
    """gemm_expert_layer on fixed buffers, validated and marshalled once."""
    args, keep = _layer_args(plan, X, ids, weights, W_up, W_down, Y, ws, base)
    return PreparedCall(load_library().gemm_expert_layer, args, keep, stream)


def _lora_args(plan, X_r, W_r, A_r, B, adapter, Y, ws, scale):
    base, keep = _ar_args(plan, X_r, W_r, Y, ws)
    M, N = Y.shape
    if len(A_r) != len(X_r):
        raise ValueError("A_r needs one tensor per shard")
    _dense(B, "B", _BF16, (None, N, None))
    L, _, rank = B.shape
    for r, a in enumerate(A_r):
        _dense(a, f"A_r[{r}]", _BF16, (L, rank, X_r[r].shape[1]))
    _dense(adapter, "adapter", torch.int32, (M,))
    if scale is not None:
        _dense(scale, "scale", torch.float32, (L,))
    ap, aa = _ptrs(A_r)
    args = base[:7] + (L, rank, ap, _ptr(B), _ptr(adapter), _ptr(scale)) + base[7:]
    return args, (keep, aa, A_r, B, adapter, scale)


def gemm_ar_lora(plan: Plan, X_r: Sequence[torch.Tensor], W_r: Sequence[torch.Tensor],
                 A_r: Sequence[torch.Tensor], B: torch.Tensor, adapter: torch.Tensor,
                 Y: torch.Tensor, ws: torch.Tensor, scale: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """gemm_ar's sum plus each row's low-rank adapter a = adapter[m] (int32; outside
    0..L-1: none): scale[a] * (sum_r X_r @ A_r[a].T) @ B[a].T (A_r: L x rank x K_r,
    B: L x N x rank, scale: fp32 or None)."""
    args, _ = _lora_args(plan, X_r, W_r, A_r, B, adapter, Y, ws, scale)
    _check(load_library().gemm_ar_lora(*args, _stream(stream)))
    return Y


def prepare_ar_lora(plan: Plan, X_r, W_r, A_r, B, adapter, Y, ws, scale=None, stream=None) -> PreparedCall:
    """gemm_ar_lora on fixed buffers, validated and marshalled once."""
    args, keep = _lora_args(plan, X_r, W_r, A_r, B, adapter, Y, ws, scale)
    return PreparedCall(load_library().gemm_ar_lora, args, keep, stream)


# ------------------------------------------------------------ 8-bit projections

_E4M3 = torch.float8_e4m3fn
SCALE_BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // SCALE_BLOCK)


def _norm_args(plan, X, gamma, eps, residual, sum, Y, Q, scale):
    _bf16_2d(X, "X")
    M, H = X.shape
    for t, name in ((residual, "residual"), (sum, "sum"), (Y, "Y")):
        if t is not None:
            _dense(t, name, _BF16, (M, H))
    if gamma is not None:
        _dense(gamma, "gamma", _BF16, (H,))
    if (Q is None) != (scale is None):
        raise ValueError("Q and scale come together")
    if Q is not None:
        _dense(Q, "Q", _E4M3, (M, H))
        _dense(scale, "scale", torch.float32, (_blocks(H), M))
    args = (plan.handle, M, H, _ptr(X), _ptr(residual), _ptr(gamma), float(eps), _ptr(sum), _ptr(Y), _ptr(Q),
            _ptr(scale))
    return args, (X, gamma, residual, sum, Y, Q, scale)


def gemm_shard_rms_norm(plan: Plan, X: torch.Tensor, gamma: Optional[torch.Tensor], eps: float,
                        residual: Optional[torch.Tensor] = None, sum: Optional[torch.Tensor] = None,
                        Y: Optional[torch.Tensor] = None, Q: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, stream=None):
    """h = X + residual; sum = h; Y = h / sqrt(mean(h^2) + eps) * gamma (M x H, bf16), and
    the same in 8 bits: Q (e4m3) with scale (ceil(H / 128) x M, fp32). Returns (sum, Y, Q,
    scale); each may be None, not all."""
    args, _ = _norm_args(plan, X, gamma, eps, residual, sum, Y, Q, scale)
    _check(load_library().gemm_shard_rms_norm(*args, _stream(stream)))
    return sum, Y, Q, scale


def prepare_rms_norm(plan: Plan, X, gamma, eps, residual=None, sum=None, Y=None, Q=None, scale=None,
                     stream=None) -> PreparedCall:
    """gemm_shard_rms_norm on fixed buffers, validated and marshalled once."""
    args, keep = _norm_args(plan, X, gamma, eps, residual, sum, Y, Q, scale)
    return PreparedCall(load_library().gemm_shard_rms_norm, args, keep, stream)


def _quantize_args(plan, X, Q, scale, block_rows):
    _bf16_2d(X, "X")
    rows, cols = X.shape
    _dense(Q, "Q", _E4M3, (rows, cols))
    _dense(scale, "scale", torch.float32,
           (_blocks(cols), rows) if int(block_rows) == 1 else (_blocks(rows), _blocks(cols)))
    args = (plan.handle, rows, cols, int(block_rows), _ptr(X), _ptr(Q), _ptr(scale))
    return args, (X, Q, scale)


def gemm_shard_quantize(plan: Plan, X: torch.Tensor, Q: torch.Tensor, scale: torch.Tensor,
                        block_rows: int = 1, stream=None):
    """X (rows x cols, bf16) in 8 bits: Q (e4m3) with a scale for each row and 128 columns
    (block_rows 1; scale: ceil(cols / 128) x rows) or for each block of 128 x 128
    (block_rows 128; scale: ceil(rows / 128) x ceil(cols / 128)). Returns (Q, scale)."""
    args, _ = _quantize_args(plan, X, Q, scale, block_rows)
    _check(load_library().gemm_shard_quantize(*args, _stream(stream)))
    return Q, scale


def prepare_quantize(plan: Plan, X, Q, scale, block_rows=1, stream=None) -> PreparedCall:
    """gemm_shard_quantize on fixed buffers, validated and marshalled once."""
    args, keep = _quantize_args(plan, X, Q, scale, block_rows)
    return PreparedCall(load_library().gemm_shard_quantize, args, keep, stream)


def _ar_fp8_args(plan, X_r, SX_r, W_r, SW_r, Y, ws):
    R = len(X_r)
    if R == 0 or not R == len(SX_r) == len(W_r) == len(SW_r):
        raise ValueError("X_r, SX_r, W_r and SW_r need the same, non-zero number of shards")
    _bf16_2d(Y, "Y")
    M, N = Y.shape
    K_r = []
    for r in range(R):
        _dense(X_r[r], f"X_r[{r}]", _E4M3, (M, None))
        k = X_r[r].shape[1]
        _dense(SX_r[r], f"SX_r[{r}]", torch.float32, (_blocks(k), M))
        _dense(W_r[r], f"W_r[{r}]", _E4M3, (N, k))
        _dense(SW_r[r], f"SW_r[{r}]", torch.float32, (_blocks(N), _blocks(k)))
        K_r.append(k)
    k, ka = _i64s(K_r)
    xp, xa = _ptrs(X_r)
    sxp, sxa = _ptrs(SX_r)
    wp, wa = _ptrs(W_r)
    swp, swa = _ptrs(SW_r)
    wsp, wsn = _ws(ws)
    args = (plan.handle, M, N, R, k, xp, sxp, wp, swp, _ptr(Y), wsp, wsn)
    return args, (ka, xa, sxa, wa, swa, X_r, SX_r, W_r, SW_r, Y, ws)


def gemm_ar_fp8(plan: Plan, X_r: Sequence[torch.Tensor], SX_r: Sequence[torch.Tensor],
                W_r: Sequence[torch.Tensor], SW_r: Sequence[torch.Tensor], Y: torch.Tensor,
                ws: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = sum_r X_r @ W_r.T over what 8-bit operands stand for (X_r: M x K_r and W_r: N x
    K_r, e4m3; SX_r: ceil(K_r / 128) x M and SW_r: ceil(N / 128) x ceil(K_r / 128), fp32;
    Y: M x N, bf16)."""
    args, _ = _ar_fp8_args(plan, X_r, SX_r, W_r, SW_r, Y, ws)
    _check(load_library().gemm_ar_fp8(*args, _stream(stream)))
    return Y


def prepare_ar_fp8(plan: Plan, X_r, SX_r, W_r, SW_r, Y, ws, stream=None) -> PreparedCall:
    """gemm_ar_fp8 on fixed buffers, validated and marshalled once."""
    args, keep = _ar_fp8_args(plan, X_r, SX_r, W_r, SW_r, Y, ws)
    return PreparedCall(load_library().gemm_ar_fp8, args, keep, stream)


def _ag_fp8_args(plan, A_r, SA_r, W, SW, Y, ws):
    R = len(A_r)
    if R == 0 or R != len(SA_r):
        raise ValueError("A_r and SA_r need the same, non-zero number of shards")
    _dense(W, "W", _E4M3, dim=2)
    N, K = W.shape
    _dense(SW, "SW", torch.float32, (_blocks(N), _blocks(K)))
    M_r = []
    for r in range(R):
        _dense(A_r[r], f"A_r[{r}]", _E4M3, (None, K))
        m = A_r[r].shape[0]
        _dense(SA_r[r], f"SA_r[{r}]", torch.float32, (_blocks(K), m))
        M_r.append(m)
    _dense(Y, "Y", _BF16, (sum(M_r), N))
    m, ma = _i64s(M_r)
    ap, aa = _ptrs([a if a.numel() else None for a in A_r])
    sp, sa = _ptrs([s if s.numel() else None for s in SA_r])
    wsp, wsn = _ws(ws)
    args = (plan.handle, N, K, R, m, ap, sp, _ptr(W), _ptr(SW), _ptr(Y), wsp, wsn)
    return args, (ma, aa, sa, A_r, SA_r, W, SW, Y, ws)


def gemm_ag_fp8(plan: Plan, A_r: Sequence[torch.Tensor], SA_r: Sequence[torch.Tensor], W: torch.Tensor,
                SW: torch.Tensor, Y: torch.Tensor, ws: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = cat(A_r) @ W.T over what 8-bit operands stand for (A_r: M_r x K and W: N x K,
    e4m3; SA_r: ceil(K / 128) x M_r and SW: ceil(N / 128) x ceil(K / 128), fp32)."""
    args, _ = _ag_fp8_args(plan, A_r, SA_r, W, SW, Y, ws)
    _check(load_library().gemm_ag_fp8(*args, _stream(stream)))
    return Y


def prepare_ag_fp8(plan: Plan, A_r, SA_r, W, SW, Y, ws, stream=None) -> PreparedCall:
    """gemm_ag_fp8 on fixed buffers, validated and marshalled once."""
    args, keep = _ag_fp8_args(plan, A_r, SA_r, W, SW, Y, ws)
    return PreparedCall(load_library().gemm_ag_fp8, args, keep, stream)
