"""Python binding of libdrgg.so, the MI355X (gfx950) ragged BF16 grouped GEMM.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI (include/drgg.h).  PyTorch supplies device memory
and the current stream.  If the library is missing the import fails loudly:
there is no fallback of any kind.

Programs (flashinfer PR #8258, opening summary paragraph), shapes row-major:

    grouped_gemm_fwd(X [M,K], W [E,N,K], offsets [E+1])   -> Y  [M,N]    = X W_e^T
    grouped_gemm_dgrad(G [M,N], W [E,N,K], offsets)       -> dX [M,K]    = G W_e
    grouped_gemm_wgrad(X [M,K], G [M,N], offsets)         -> dW [E,N,K]  = G_e^T X_e
    router_gemm_fp32_bf16x3(X [M,K] fp32, Wr [N,K] fp32)  -> out [M,N] fp32

Around them, for a whole expert layer: the router's selection (moe_route,
moe_route_grad), the movement of rows (moe_dispatch, moe_combine,
moe_combine_grad), and products in 8-bit integers (quantize_int8,
grouped_gemm_int8, gemm_int8); moe_ffn_int8 runs them as one serving block, and
`moe` holds the differentiable ones.  moe_route_scores selects by sigmoid or
softmax scores with a bias and groups of experts; quantize_mxfp4,
grouped_gemm_mxfp4, gemm_mxfp4 and moe_ffn_mxfp4 are the products and the serving
block in microscaled 4-bit floating point; moe_gate_int8 is a training step's gated
activation, which keeps its inputs in 8 bits for its gradient.

``offsets`` is an int32 CUDA tensor: offsets[0] = 0, non-decreasing,
offsets[E] = M; expert e owns tokens offsets[e] .. offsets[e+1]-1.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdrgg.so")

BF16, FP32 = 0, 1
OP_FWD, OP_DGRAD, OP_WGRAD = 0, 1, 2
KNOB_TILE, KNOB_GRID, KNOB_REVERSE, KNOB_TIMING, KNOB_NONDET = 1, 2, 3, 4, 5
KNOB_CHECK_OFFSETS, KNOB_CHECK_WORKSPACE, KNOB_DELAY_SEED, KNOB_SPLIT_REPORT = 6, 7, 8, 9
KNOB_DGRAD_WT = 10
TILE_AUTO, TILE_256x256, TILE_128x128, TILE_256x128, TILE_128x256, TILE_64x256 = range(6)

# the symbols include/drgg.h declares
EXPORTS = (
    "grouped_gemm_fwd", "grouped_gemm_dgrad", "grouped_gemm_wgrad", "router_gemm_fp32_bf16x3",
    "router_gemm_fp32_bf16x3_ws", "router_workspace_size", "drgg_router_split",
    "batched_gemm_fwd", "batched_gemm_dgrad", "batched_gemm_wgrad",
    "drgg_route_split", "drgg_route_clear", "drgg_route_count", "drgg_hold_cus",
    "grouped_gemm_workspace_size", "drgg_workspace_init", "drgg_plan", "drgg_wgrad_chunking",
    "drgg_tailsplit_units", "drgg_wgrad_tail_plan", "drgg_wgrad_split_plan", "grouped_gemm_wgrad_noalloc",
    "drgg_set_knob", "drgg_timing_count", "drgg_timing_read", "drgg_status_string", "drgg_abi_version",
    "moe_route", "moe_route_workspace_size", "moe_route_grad", "moe_dispatch", "moe_combine", "moe_combine_grad",
    "quantize_int8", "grouped_gemm_int8", "gemm_int8", "moe_ffn_int8", "moe_ffn_int8_workspace_size",
    "moe_route_scores", "moe_route_scores_grad", "quantize_mxfp4", "dequantize_mxfp4", "grouped_gemm_mxfp4",
    "gemm_mxfp4", "moe_ffn_mxfp4", "moe_ffn_mxfp4_workspace_size", "moe_gate_int8", "moe_gate_int8_grad",
)


class DrggError(RuntimeError):
    """A non-zero status from the C ABI; the message is drgg_status_string."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
        ("mfma_m", ctypes.c_int32), ("mfma_n", ctypes.c_int32), ("mfma_k", ctypes.c_int32),
        ("grid", ctypes.c_int64), ("chunk_max", ctypes.c_int64), ("unit", ctypes.c_int64),
        ("max_partials", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class Batched(ctypes.Structure):
    """drgg_batched: shape and element strides of a batched call."""
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_row", ctypes.c_int64), ("a_batch", ctypes.c_int64),
        ("b_row", ctypes.c_int64), ("b_batch", ctypes.c_int64),
        ("o_row", ctypes.c_int64), ("o_batch", ctypes.c_int64),
    ]


class ScoringStruct(ctypes.Structure):
    """drgg_scoring."""
    _fields_ = [
        ("score", ctypes.c_int), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("best", ctypes.c_int32),
        ("renormalize", ctypes.c_int), ("scale", ctypes.c_float), ("bias", ctypes.c_void_p),
    ]


def _load(path=LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python -m dense_ragged_grouped_amd.build` "
            "(the grouped GEMM has no fallback path)")
    # One HIP runtime per process: libdrgg.so needs libamdhip64.so.7, which
    # resolves to the runtime already loaded under that name.  torch bundles
    # its own; loaded first, it serves both.  Loaded after this library (whose
    # runpath finds the system runtime), torch would bring a second HIP/HSA
    # runtime, and the one initialised last finds no device.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz, c_int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    gemm = [vp, vp, vp, i32, i64, i64, i64, c_int, c_int, vp, vp, sz, vp]
    for name in ("grouped_gemm_fwd", "grouped_gemm_dgrad", "grouped_gemm_wgrad"):
        getattr(lib, name).argtypes = gemm
        getattr(lib, name).restype = c_int
    lib.grouped_gemm_wgrad_noalloc.argtypes = [vp, vp, vp, i32, i64, i64, i64, c_int, c_int, vp, vp]
    lib.grouped_gemm_wgrad_noalloc.restype = c_int
    pb = ctypes.POINTER(Batched)
    lib.batched_gemm_fwd.argtypes = [vp, vp, pb, c_int, vp, vp]
    lib.batched_gemm_dgrad.argtypes = [vp, vp, pb, c_int, vp, vp, sz, vp]
    lib.batched_gemm_wgrad.argtypes = [vp, vp, pb, c_int, c_int, vp, vp, sz, vp]
    for name in ("batched_gemm_fwd", "batched_gemm_dgrad", "batched_gemm_wgrad"):
        getattr(lib, name).restype = c_int
    lib.router_gemm_fp32_bf16x3.argtypes = [vp, vp, i64, i64, i64, vp, vp]
    lib.router_gemm_fp32_bf16x3.restype = c_int
    lib.router_gemm_fp32_bf16x3_ws.argtypes = [vp, vp, i64, i64, i64, vp, vp, sz, vp]
    lib.router_gemm_fp32_bf16x3_ws.restype = c_int
    lib.router_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    lib.router_workspace_size.restype = c_int
    lib.drgg_router_split.argtypes = [i64, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.drgg_router_split.restype = c_int
    lib.grouped_gemm_workspace_size.argtypes = [c_int, i32, i64, i64, i64, c_int, c_int, c_int,
                                                ctypes.POINTER(sz)]
    lib.grouped_gemm_workspace_size.restype = c_int
    lib.drgg_workspace_init.argtypes = [vp, sz, vp]
    lib.drgg_workspace_init.restype = c_int
    lib.drgg_plan.argtypes = [c_int, i32, i64, i64, i64, c_int, c_int, c_int, ctypes.POINTER(PlanInfo)]
    lib.drgg_plan.restype = c_int
    lib.drgg_wgrad_chunking.argtypes = [i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.drgg_wgrad_chunking.restype = c_int
    lib.drgg_wgrad_tail_plan.argtypes = [vp, i32, i64, i64, ctypes.POINTER(c_int), vp]
    lib.drgg_wgrad_tail_plan.restype = c_int
    lib.drgg_wgrad_split_plan.argtypes = [vp, i32, i64, i64, c_int, i64, ctypes.POINTER(c_int), ctypes.POINTER(i64),
                                          ctypes.POINTER(c_int)]
    lib.drgg_wgrad_split_plan.restype = c_int
    lib.drgg_tailsplit_units.argtypes = [i64, i64, ctypes.POINTER(i64)]
    lib.drgg_tailsplit_units.restype = c_int
    lib.drgg_route_split.argtypes = [i32, i64, i64, i64, c_int]
    lib.drgg_route_split.restype = c_int
    lib.drgg_hold_cus.argtypes = [c_int, i64, vp]
    lib.drgg_hold_cus.restype = c_int
    lib.drgg_route_clear.argtypes = []
    lib.drgg_route_clear.restype = c_int
    lib.drgg_route_count.argtypes = []
    lib.drgg_route_count.restype = c_int
    lib.drgg_set_knob.argtypes = [c_int, i64]
    lib.drgg_set_knob.restype = c_int
    lib.drgg_timing_count.argtypes = []
    lib.drgg_timing_count.restype = c_int
    lib.drgg_timing_read.argtypes = [c_int, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float)]
    lib.drgg_timing_read.restype = c_int
    lib.moe_route.argtypes = [vp, i64, i32, i32, c_int, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_route_workspace_size.argtypes = [i64, i32, i32, ctypes.POINTER(sz)]
    lib.moe_route_grad.argtypes = [vp, vp, vp, vp, i64, i32, i32, c_int, vp, vp]
    lib.moe_dispatch.argtypes = [vp, vp, i64, i32, i64, c_int, vp, vp]
    lib.moe_combine.argtypes = [vp, vp, vp, i64, i32, i64, c_int, vp, vp]
    lib.moe_combine_grad.argtypes = [vp, vp, vp, vp, i64, i32, i64, c_int, vp, vp, vp]
    lib.quantize_int8.argtypes = [vp, c_int, i64, i64, vp, i32, vp, vp, vp]
    lib.grouped_gemm_int8.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, i64, c_int, c_int, vp, vp]
    lib.gemm_int8.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, c_int, vp, vp]
    lib.moe_ffn_int8.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, i64, c_int, vp, vp, sz, vp]
    lib.moe_ffn_int8_workspace_size.argtypes = [i64, i32, i32, i64, i64, ctypes.POINTER(sz)]
    ps = ctypes.POINTER(ScoringStruct)
    lib.moe_route_scores.argtypes = [vp, i64, i32, i32, ps, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_route_scores_grad.argtypes = [vp, vp, vp, vp, i64, i32, i32, ps, vp, vp]
    lib.quantize_mxfp4.argtypes = [vp, c_int, i64, i64, vp, vp, vp]
    lib.dequantize_mxfp4.argtypes = [vp, vp, i64, i64, c_int, vp, vp]
    lib.grouped_gemm_mxfp4.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, i64, c_int, c_int, vp, vp]
    lib.gemm_mxfp4.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, c_int, vp, vp]
    lib.moe_ffn_mxfp4.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, i64, ps, vp, vp, sz, vp]
    lib.moe_ffn_mxfp4_workspace_size.argtypes = [i64, i32, i32, i64, i64, ctypes.POINTER(sz)]
    lib.moe_gate_int8.argtypes = [vp, vp, vp, i64, i32, i64, vp, vp, vp, vp]
    lib.moe_gate_int8_grad.argtypes = [vp, vp, vp, vp, vp, i64, i32, i64, vp, vp, vp, vp]
    for name in EXPORTS[-10:]:
        getattr(lib, name).restype = c_int
    for name in ("moe_ffn_int8", "moe_ffn_int8_workspace_size", "moe_route", "moe_route_workspace_size", "moe_route_grad", "moe_dispatch", "moe_combine",
                 "moe_combine_grad", "quantize_int8", "grouped_gemm_int8", "gemm_int8"):
        getattr(lib, name).restype = c_int
    lib.drgg_status_string.argtypes = [c_int]
    lib.drgg_status_string.restype = ctypes.c_char_p
    lib.drgg_abi_version.argtypes = []
    lib.drgg_abi_version.restype = c_int
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.drgg_status_string(status).decode()


def abi_version() -> int:
    return lib.drgg_abi_version()


def _check(status: int, where: str):
    if status != 0:
        raise DrggError(status, where)


# ---- host-only queries ------------------------------------------------------

def plan(op: int, E: int, M: int, N: int, K: int, out_dtype: int = BF16, deterministic: bool = True,
         cu_count: int = 256) -> dict:
    """The plan a call would use (no GPU needed when cu_count > 0)."""
    info = PlanInfo()
    _check(lib.drgg_plan(op, E, M, N, K, out_dtype, int(bool(deterministic)), cu_count, ctypes.byref(info)),
           "drgg_plan")
    return info.as_dict()


def wgrad_chunking(T: int, chunk_max: int):
    """(chunk length, chunk count) of an expert with T tokens."""
    ln, n = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.drgg_wgrad_chunking(T, chunk_max, ctypes.byref(ln), ctypes.byref(n)), "drgg_wgrad_chunking")
    return ln.value, n.value


def tailsplit_units(tiles: int, workers: int):
    """(tiles, units, full, split) of the tail-split rule: `tiles` equal
    tiles on `workers` persistent workers; a partial last wave of
    tail = tiles mod workers tiles is cut into 2 * tail half units when that
    fits one wave, else every tile stays whole."""
    out = (ctypes.c_int64 * 4)()
    _check(lib.drgg_tailsplit_units(int(tiles), int(workers), out), "drgg_tailsplit_units")
    return tuple(int(v) for v in out)


def wgrad_tail_plan(offsets, N: int, K: int):
    """(tail_only, row0) of the deterministic weight gradient's plan for host
    group offsets (a sequence of E + 1 ints): whether the kernel runs the
    tail-only plan, and per expert the first dW row that comes from folded
    partials (the rows above it are whole tiles, stored directly)."""
    import numpy as np
    o = np.ascontiguousarray(np.asarray(offsets, dtype=np.int32))
    E = o.size - 1
    tail = ctypes.c_int()
    row0 = np.zeros(max(E, 1), dtype=np.int32)
    _check(lib.drgg_wgrad_tail_plan(o.ctypes.data, E, N, K, ctypes.byref(tail), row0.ctypes.data),
           "drgg_wgrad_tail_plan")
    return bool(tail.value), row0[:E]


def wgrad_split_plan(offsets, N: int, K: int, grid: int = 256, tile: int = 0, banded: bool = False):
    """(slack, tail_tiles) of the split program's walk for host group offsets
    on `grid` workgroups: whether its tail tiles run whole on the
    least-loaded workgroups (slack placement), and how many tail tiles the
    banded walk has; with banded=True also whether the banded walk runs."""
    import numpy as np
    o = np.ascontiguousarray(np.asarray(offsets, dtype=np.int32))
    slack, tail, band = ctypes.c_int(), ctypes.c_int64(), ctypes.c_int()
    _check(lib.drgg_wgrad_split_plan(o.ctypes.data, o.size - 1, N, K, tile, grid, ctypes.byref(slack),
                                     ctypes.byref(tail), ctypes.byref(band)), "drgg_wgrad_split_plan")
    if banded:
        return bool(slack.value), int(tail.value), bool(band.value)
    return bool(slack.value), int(tail.value)


def wgrad_runs_deterministic(E: int, M: int, N: int, K: int, out_dtype: int = BF16,
                             deterministic: bool = True) -> bool:
    """Whether a weight-gradient call runs the deterministic program: always
    for deterministic=True; for deterministic=False unless the route table
    (or KNOB_NONDET) sends the point to the split program."""
    if deterministic:
        return True
    return plan(OP_WGRAD, E, M, N, K, out_dtype, False, 1)["unit"] == 0


def route_split(E: int, M: int, N: int, K: int, out_dtype: int = BF16):
    """Send non-deterministic weight-gradient calls at this exact point to the
    split program (see load_routes)."""
    _check(lib.drgg_route_split(E, M, N, K, out_dtype), "drgg_route_split")


def hold_cus(cus: int, microseconds: int, stream=None):
    """Calibration aid: occupy `cus` compute units for `microseconds` on
    `stream` (default: the current stream)."""
    torch = _torch()
    _check(lib.drgg_hold_cus(int(cus), int(microseconds), _stream(torch.device("cuda"), stream)), "drgg_hold_cus")


def route_clear():
    _check(lib.drgg_route_clear(), "drgg_route_clear")


def route_count() -> int:
    return lib.drgg_route_count()


DEFAULT_ROUTES = os.path.join(os.path.dirname(os.path.abspath(__file__)), "routes_mi355x.json")


def load_default_routes() -> int:
    """Install the route table measured on MI355X (256 CUs) that ships with
    the package (done at import unless DRGG_NO_ROUTES=1)."""
    return load_routes(DEFAULT_ROUTES) if os.path.exists(DEFAULT_ROUTES) else 0


def load_routes(path: str) -> int:
    """Install the split points of a route table written by
    `python -m dense_ragged_grouped_amd.calibrate` (JSON); returns how many.
    The table applies to the kind of device it was measured on."""
    import json
    with open(path) as f:
        table = json.load(f)
    n = 0
    for pt in table.get("points", []):
        if pt.get("program") == "split":
            route_split(pt["E"], pt["M"], pt["N"], pt["K"], pt.get("out_dtype", BF16))
            n += 1
    return n


def set_knob(knob: int, value: int):
    """Test knobs (tile shape, persistent grid, reverse walk, timing, split
    program for non-deterministic weight gradients, the debug checks of the
    offsets and of the split program's workspace); 0 restores the default."""
    _check(lib.drgg_set_knob(knob, int(value)), "drgg_set_knob")


def last_call_kernel_times():
    """With KNOB_TIMING on: [(kernel name, milliseconds)] of the most recent
    call's kernel launches, timed by HIP events on the launch stream."""
    out = []
    for i in range(lib.drgg_timing_count()):
        name, ms = ctypes.c_char_p(), ctypes.c_float()
        _check(lib.drgg_timing_read(i, ctypes.byref(name), ctypes.byref(ms)), "drgg_timing_read")
        out.append((name.value.decode(), ms.value))
    return out


def workspace_size(op: int, E: int, M: int, N: int, K: int, out_dtype: int = BF16,
                   deterministic: bool = True, cu_count: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(lib.grouped_gemm_workspace_size(op, E, M, N, K, out_dtype, int(bool(deterministic)), cu_count,
                                           ctypes.byref(n)), "grouped_gemm_workspace_size")
    return n.value


# ---- torch marshalling ---------------------------------------------------------

try:
    import torch as _torch_module
except ImportError:   # the host-only queries work without it
    _torch_module = None


def _torch():
    if _torch_module is None:
        raise ImportError("this call needs torch")
    return _torch_module


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt in (torch.bfloat16, BF16, "bf16"):
        return BF16
    if dt in (torch.float32, FP32, "fp32"):
        return FP32
    raise ValueError(f"unsupported output dtype {dt!r}")


def _torch_dtype(code: int):
    torch = _torch()
    return torch.bfloat16 if code == BF16 else torch.float32


def _need(t, dtype, name, ndim):
    if not isinstance(t, _torch_module.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def _stream(device, stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _on_one_device(stream, *tensors):
    """Check that the tensors of one call (None entries skipped) and the
    stream, if given, are on one device, and return a context that makes
    that device current for the launch (the library plans for, and launches
    on, the current device)."""
    torch = _torch()
    dev = tensors[0].device
    for t in tensors[1:]:
        if t is not None and t.device != dev:
            raise ValueError(f"the tensors of one call must be on one device ({dev} and {t.device})")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.device(dev)


def _new(shape, dtype, like, stream):
    """A result of a call on `stream`, on the device of `like`.  Allocated on
    the stream that writes it: memory that is free on the caller's stream may
    still be in use there.  Recorded on the caller's stream, which will read
    it: dropped, it is not handed out again before that has happened."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    torch = _torch()
    caller = torch.cuda.current_stream(like.device)
    if stream == caller:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(caller)
    return t


class Workspace:
    """Device workspace for the weight gradient, grown on demand.

    Allocated and zeroed on the stream of the call that needs it (so the
    zeroing is ordered before that call's kernels, and torch's allocator
    ties the memory to that stream); used on another stream, the buffer is
    recorded on it, so that a buffer replaced by a larger one is not handed
    out again before the calls using it have finished.  The split program
    leaves its tile sums and tickets zero after every call, so the buffer
    stays valid for later calls.  One Workspace must not serve two calls in
    flight on different streams at once.
    """

    def __init__(self, device=None):
        torch = _torch()
        self.device = torch.device(device if device is not None else "cuda")
        self.buf = None
        self.home = None

    def get(self, nbytes: int, stream=None):
        torch = _torch()
        if nbytes == 0:
            return None
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if self.buf is None or self.buf.numel() < nbytes:
            with torch.cuda.stream(s):
                self.buf = torch.zeros(nbytes + 256, dtype=torch.uint8, device=self.device)
            self.home = s
        elif s != self.home:
            self.buf.record_stream(s)
        return self.buf


# Default workspaces, one per (device, stream, program): a deterministic call
# leaves its FP32 partials in the buffer, while the split program needs its
# tile sums and tickets to be zero, so the two never share a buffer; calls on
# different streams may run at the same time, so they never share one either.
_default_ws = {}


def _need_span(workspace):
    """A workspace's size in bytes is that of its elements: an expanded tensor
    has fewer."""
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")


def _workspace(device, nbytes, workspace, deterministic, kind="wgrad", stream=None):
    torch = _torch()
    if workspace is False:   # explicitly none (the data gradient's direct program)
        return None, 0
    s = stream if stream is not None else torch.cuda.current_stream(device)
    if workspace is not None:
        buf = workspace.get(nbytes, s) if isinstance(workspace, Workspace) else workspace
        if buf is not None and buf.device != device:
            raise ValueError(f"the workspace is on {buf.device}, the operands on {device}")
        if buf is not None:
            _need_span(buf)
    else:
        # keyed by the program that runs (`deterministic` here: whether the
        # deterministic program runs): a non-deterministic call routed to it
        # shares its buffer of partials, the split program has its own,
        # zeroed one; the data gradient's W^T and the router's reduction
        # slices have their own
        prog = kind if kind in ("dgrad", "router") else bool(deterministic)
        key = (str(device), s.cuda_stream, prog)
        if key not in _default_ws:
            _default_ws[key] = Workspace(device)
        buf = _default_ws[key].get(nbytes, s)
    if buf is None:
        return None, 0
    return ctypes.c_void_p(buf.data_ptr()), buf.numel() * buf.element_size()


def _offsets(offsets):
    torch = _torch()
    _need(offsets, torch.int32, "group_offsets", 1)
    return offsets.numel() - 1


def grouped_gemm_fwd(X, W, group_offsets, out_dtype=None, deterministic=True, out=None, stream=None):
    """Y[t] = X[t] W[e(t)]^T with FP32 accumulation; out_dtype bf16 (default) or fp32."""
    torch = _torch()
    _need(X, torch.bfloat16, "X", 2)
    _need(W, torch.bfloat16, "W", 3)
    E = _offsets(group_offsets)
    M, K = X.shape
    En, N, Kw = W.shape
    if En != E or Kw != K:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, E={E}")
    code = _dtype_code(out_dtype if out_dtype is not None else torch.bfloat16)
    if out is None:
        out = _new((M, N), _torch_dtype(code), X, stream)
    else:
        _need(out, _torch_dtype(code), "out", 2)
        if tuple(out.shape) != (M, N):
            raise ValueError("out has the wrong shape")
    with _on_one_device(stream, X, W, group_offsets, out):
        st = lib.grouped_gemm_fwd(X.data_ptr(), W.data_ptr(), group_offsets.data_ptr(), E, M, N, K, code,
                                  int(bool(deterministic)), out.data_ptr(), None, 0, _stream(X.device, stream))
    _check(st, "grouped_gemm_fwd")
    return out


def grouped_gemm_dgrad(G, W, group_offsets, out_dtype=None, deterministic=True, out=None, workspace=None,
                       stream=None):
    """dX[t] = G[t] W[e(t)] with FP32 accumulation.  `workspace` (a Workspace,
    a device tensor, None for the default buffer, or False for none) holds
    W^T, which makes the product faster when the experts average at least
    3072 tokens (below that no W^T is made and the default buffer is not
    allocated); the result is bitwise the same either way."""
    torch = _torch()
    _need(G, torch.bfloat16, "G", 2)
    _need(W, torch.bfloat16, "W", 3)
    E = _offsets(group_offsets)
    M, N = G.shape
    En, Nw, K = W.shape
    if En != E or Nw != N:
        raise ValueError(f"shape mismatch: G {tuple(G.shape)}, W {tuple(W.shape)}, E={E}")
    code = _dtype_code(out_dtype if out_dtype is not None else torch.bfloat16)
    if out is None:
        out = _new((M, K), _torch_dtype(code), G, stream)
    else:
        _need(out, _torch_dtype(code), "out", 2)
        if tuple(out.shape) != (M, K):
            raise ValueError("out has the wrong shape")
    nbytes = workspace_size(OP_DGRAD, E, M, N, K, code, deterministic)
    with _on_one_device(stream, G, W, group_offsets, out):
        ws_ptr, ws_bytes = _workspace(G.device, nbytes, workspace, deterministic, kind="dgrad", stream=stream)
        st = lib.grouped_gemm_dgrad(G.data_ptr(), W.data_ptr(), group_offsets.data_ptr(), E, M, N, K, code,
                                    int(bool(deterministic)), out.data_ptr(), ws_ptr, ws_bytes,
                                    _stream(G.device, stream))
    _check(st, "grouped_gemm_dgrad")
    return out


def grouped_gemm_wgrad(X, G, group_offsets, out_dtype=None, deterministic=True, out=None, workspace=None,
                       stream=None):
    """dW[e] = G_e^T X_e over each expert's tokens (+0 for experts without tokens)."""
    torch = _torch()
    _need(X, torch.bfloat16, "X", 2)
    _need(G, torch.bfloat16, "G", 2)
    E = _offsets(group_offsets)
    M, K = X.shape
    Mg, N = G.shape
    if Mg != M:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, G {tuple(G.shape)}")
    code = _dtype_code(out_dtype if out_dtype is not None else torch.bfloat16)
    if out is None:
        out = _new((E, N, K), _torch_dtype(code), X, stream)
    else:
        _need(out, _torch_dtype(code), "out", 3)
        if tuple(out.shape) != (E, N, K):
            raise ValueError("out has the wrong shape")
    nbytes = workspace_size(OP_WGRAD, E, M, N, K, code, deterministic)
    with _on_one_device(stream, X, G, group_offsets, out):
        ws_ptr, ws_bytes = _workspace(X.device, nbytes, workspace,
                                      wgrad_runs_deterministic(E, M, N, K, code, deterministic), stream=stream)
        st = lib.grouped_gemm_wgrad(X.data_ptr(), G.data_ptr(), group_offsets.data_ptr(), E, M, N, K, code,
                                    int(bool(deterministic)), out.data_ptr(), ws_ptr, ws_bytes,
                                    _stream(X.device, stream))
    _check(st, "grouped_gemm_wgrad")
    return out


def grouped_gemm_wgrad_noalloc(X, G, group_offsets, out, deterministic=True, stream=None):
    """grouped_gemm_wgrad into a caller-given `out` [E, N, K] (BF16 or FP32)
    with the library's fixed per-device workspace: the call allocates
    nothing (for code that must not, e.g. under graph capture).  Problems
    whose workspace exceeds that array (64 MiB) are refused; calls that
    overlap on one device race on it."""
    torch = _torch()
    _need(X, torch.bfloat16, "X", 2)
    _need(G, torch.bfloat16, "G", 2)
    E = _offsets(group_offsets)
    M, K = X.shape
    Mg, N = G.shape
    if Mg != M:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, G {tuple(G.shape)}")
    code = _dtype_code(out.dtype)
    _need(out, _torch_dtype(code), "out", 3)
    if tuple(out.shape) != (E, N, K):
        raise ValueError("out has the wrong shape")
    with _on_one_device(stream, X, G, group_offsets, out):
        st = lib.grouped_gemm_wgrad_noalloc(X.data_ptr(), G.data_ptr(), group_offsets.data_ptr(), E, M, N, K, code,
                                            int(bool(deterministic)), out.data_ptr(), _stream(X.device, stream))
    _check(st, "grouped_gemm_wgrad_noalloc")
    return out


# ---- batched calls: [B, T, row] views with any batch and row strides -----------

def _need_rows(t, name, shape=None):
    """A BF16 CUDA tensor [B, T, row] whose rows are contiguous (any batch
    and row strides, e.g. a transposed head-interleaved [T, B, row])."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError(f"{name} must be a 3-d tensor with contiguous rows")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _out_rows(out, shape, code, like, stream, name="out"):
    if out is None:
        return _new(shape, _torch_dtype(code), like, stream)
    if out.dtype != _torch_dtype(code):
        raise TypeError(f"{name} must be {_torch_dtype(code)}")
    _need_rows(out, name, shape)
    return out


def batched_gemm_fwd(X, W, out_dtype=None, out=None, stream=None):
    """Y[b] = X[b] W[b]^T for b < B: X [B, T, K] (rows contiguous, any
    strides, e.g. a head-interleaved [T, H, K] activation passed as
    X.transpose(0, 1)), W [B, N, K] contiguous; Y [B, T, N] (new and
    contiguous, or `out` with contiguous rows)."""
    torch = _torch()
    _need_rows(X, "X")
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    _need(W, torch.bfloat16, "W", 3)
    B, T, K = X.shape
    if W.shape[0] != B or W.shape[2] != K:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    N = W.shape[1]
    code = _dtype_code(out_dtype if out_dtype is not None else torch.bfloat16)
    out = _out_rows(out, (B, T, N), code, X, stream)
    b = Batched(B, T, N, K, X.stride(1), X.stride(0), 0, 0, out.stride(1), out.stride(0))
    with _on_one_device(stream, X, W, out):
        st = lib.batched_gemm_fwd(X.data_ptr(), W.data_ptr(), ctypes.byref(b), code, out.data_ptr(),
                                  _stream(X.device, stream))
    _check(st, "batched_gemm_fwd")
    return out


def batched_gemm_dgrad(G, W, out_dtype=None, out=None, workspace=None, stream=None):
    """dX[b] = G[b] W[b]: G [B, T, N] (rows contiguous), W [B, N, K]
    contiguous; dX [B, T, K].  `workspace` as for grouped_gemm_dgrad."""
    torch = _torch()
    _need_rows(G, "G")
    if G.dtype != torch.bfloat16:
        raise TypeError("G must be bfloat16")
    _need(W, torch.bfloat16, "W", 3)
    B, T, N = G.shape
    if W.shape[0] != B or W.shape[1] != N:
        raise ValueError(f"shape mismatch: G {tuple(G.shape)}, W {tuple(W.shape)}")
    K = W.shape[2]
    code = _dtype_code(out_dtype if out_dtype is not None else torch.bfloat16)
    out = _out_rows(out, (B, T, K), code, G, stream)
    nbytes = workspace_size(OP_DGRAD, B, B * T, N, K, code, True)
    b = Batched(B, T, N, K, G.stride(1), G.stride(0), 0, 0, out.stride(1), out.stride(0))
    with _on_one_device(stream, G, W, out):
        ws_ptr, ws_bytes = _workspace(G.device, nbytes, workspace, True, kind="dgrad", stream=stream)
        st = lib.batched_gemm_dgrad(G.data_ptr(), W.data_ptr(), ctypes.byref(b), code, out.data_ptr(), ws_ptr,
                                    ws_bytes, _stream(G.device, stream))
    _check(st, "batched_gemm_dgrad")
    return out


def batched_gemm_wgrad(X, G, out_dtype=None, deterministic=True, out=None, workspace=None, stream=None):
    """dW[b] = G[b]^T X[b]: X [B, T, K], G [B, T, N] (rows contiguous, any
    strides); dW [B, N, K] contiguous.  Workspace as for grouped_gemm_wgrad
    with E = B, M = B*T."""
    torch = _torch()
    _need_rows(X, "X")
    _need_rows(G, "G")
    if X.dtype != torch.bfloat16 or G.dtype != torch.bfloat16:
        raise TypeError("X and G must be bfloat16")
    B, T, K = X.shape
    if G.shape[0] != B or G.shape[1] != T:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, G {tuple(G.shape)}")
    N = G.shape[2]
    code = _dtype_code(out_dtype if out_dtype is not None else torch.bfloat16)
    if out is None:
        out = _new((B, N, K), _torch_dtype(code), X, stream)
    else:
        _need(out, _torch_dtype(code), "out", 3)
        if tuple(out.shape) != (B, N, K):
            raise ValueError("out has the wrong shape")
    nbytes = workspace_size(OP_WGRAD, B, B * T, N, K, code, deterministic)
    b = Batched(B, T, N, K, X.stride(1), X.stride(0), G.stride(1), G.stride(0), 0, 0)
    with _on_one_device(stream, X, G, out):
        ws_ptr, ws_bytes = _workspace(X.device, nbytes, workspace,
                                      wgrad_runs_deterministic(B, B * T, N, K, code, deterministic), stream=stream)
        st = lib.batched_gemm_wgrad(X.data_ptr(), G.data_ptr(), ctypes.byref(b), code, int(bool(deterministic)),
                                    out.data_ptr(), ws_ptr, ws_bytes, _stream(X.device, stream))
    _check(st, "batched_gemm_wgrad")
    return out


def router_split(M: int, N: int, K: int):
    """(slices, values per slice) of the router call: (0, K) for the
    single-pass program."""
    ks, kq = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.drgg_router_split(M, N, K, ctypes.byref(ks), ctypes.byref(kq)), "drgg_router_split")
    return ks.value, kq.value


def router_workspace_size(M: int, N: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.router_workspace_size(M, N, K, ctypes.byref(n)), "router_workspace_size")
    return n.value


def router_gemm_fp32_bf16x3(X, Wr, out=None, stream=None, workspace=None):
    """FP32 router GEMM out = X Wr^T on BF16 MFMA via the BF16x3 split, in
    the program router_split(M, N, K) names (single pass, or reduction slices
    added in a fixed order).  `workspace` (a Workspace, a device tensor, or
    None for the default buffer) holds the slices; False always runs the
    single-pass program (no workspace)."""
    torch = _torch()
    _need(X, torch.float32, "X", 2)
    _need(Wr, torch.float32, "Wr", 2)
    M, K = X.shape
    N, Kw = Wr.shape
    if Kw != K:
        raise ValueError("shape mismatch")
    if out is None:
        out = _new((M, N), torch.float32, X, stream)
    else:
        _need(out, torch.float32, "out", 2)
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
    with _on_one_device(stream, X, Wr, out):
        if workspace is False:
            st = lib.router_gemm_fp32_bf16x3(X.data_ptr(), Wr.data_ptr(), M, N, K, out.data_ptr(),
                                             _stream(X.device, stream))
            _check(st, "router_gemm_fp32_bf16x3")
            return out
        nbytes = router_workspace_size(M, N, K)
        ws_ptr, ws_bytes = _workspace(X.device, nbytes, workspace, True, kind="router", stream=stream)
        st = lib.router_gemm_fp32_bf16x3_ws(X.data_ptr(), Wr.data_ptr(), M, N, K, out.data_ptr(), ws_ptr, ws_bytes,
                                            _stream(X.device, stream))
    _check(st, "router_gemm_fp32_bf16x3_ws")
    return out


def workspace_init(buf, stream=None):
    """Zero a workspace tensor with the library's fill kernel."""
    _need_span(buf)
    _check(lib.drgg_workspace_init(buf.data_ptr(), buf.numel() * buf.element_size(),
                                   _stream(buf.device, stream)), "drgg_workspace_init")


# ---- the operators around the grouped products ---------------------------------

class Routing(NamedTuple):
    """What moe_route returns."""
    experts: "torch.Tensor"         # [T, k] int32, largest logit first
    weights: "torch.Tensor"         # [T, k] float32
    group_offsets: "torch.Tensor"   # [E+1] int32, as the grouped products take them
    positions: "torch.Tensor"       # [T, k] int32, each pair's row in the grouped order
    tokens: "torch.Tensor"          # [T*k] int32, each row's token


def _call(name, stream, tensors, *args):
    """lib.<name>(*args, stream) on the device of `tensors` (None entries
    skipped).  These calls are short, so the usual case -- the tensors on the
    current device, its current stream -- reads the stream's handle directly
    (torch's accessors, 0.1 us each; the Stream object and the device guard
    cost 3 us)."""
    if stream is None and _RAW_STREAM:
        index = _torch_module._C._cuda_getDevice()
        for t in tensors:
            if t is not None and t.get_device() != index:
                break
        else:
            st = getattr(lib, name)(*args, _torch_module._C._cuda_getCurrentRawStream(index))
            if st:
                raise DrggError(st, name)
            return
    with _on_one_device(stream, *tensors):
        _check(getattr(lib, name)(*args, _stream(tensors[0].device, stream)), name)


def _raw_stream_accessors():
    C = getattr(_torch_module, "_C", None)
    return hasattr(C, "_cuda_getCurrentRawStream") and hasattr(C, "_cuda_getDevice")


_RAW_STREAM = _raw_stream_accessors()


def _need_shape(t, dtype, shape, name):
    _need(t, dtype, name, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _out(out, dtype, shape, like, stream):
    if out is None:
        return _new(shape, dtype, like, stream)
    _need_shape(out, dtype, shape, "out")
    return out


def _row_code(t, name):
    """The dtype code of a contiguous 2-d row tensor, BF16 or FP32."""
    torch = _torch_module
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{name} must be a bfloat16 or float32 CUDA tensor")
    _need(t, t.dtype, name, 2)
    return BF16 if t.dtype == torch.bfloat16 else FP32


def route_workspace_size(T: int, E: int, k: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.moe_route_workspace_size(T, E, k, ctypes.byref(n)), "moe_route_workspace_size")
    return n.value


def moe_route(logits, k, renormalize=True, workspace=None, stream=None):
    """The k largest of each token's router logits [T, E] (FP32; ties to the
    lowest index), their softmax weights (over the chosen, or over all experts
    with renormalize=False), and the stable grouping of the T*k pairs by
    expert, as a Routing.  A masked (-inf) logit gets weight 0, also when all
    of a token's are."""
    torch = _torch_module
    _need(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    k = int(k)
    nbytes = route_workspace_size(T, E, k)
    R = T * k
    weights = _new((T, k), torch.float32, logits, stream)
    # one allocation for the integers (four would cost three times as much)
    ints = _new((3 * R + E + 1,), torch.int32, logits, stream)
    experts, positions = ints.as_strided((T, k), (k, 1)), ints.as_strided((T, k), (k, 1), R)
    tokens, offsets = ints.as_strided((R,), (1,), 2 * R), ints.as_strided((E + 1,), (1,), 3 * R)
    ws_ptr, ws_bytes = None, 0
    if nbytes and workspace is None:
        scratch = _scratch(logits, nbytes, stream)
        ws_ptr, ws_bytes = scratch.data_ptr(), nbytes
    elif nbytes:
        ws_ptr, ws_bytes = _workspace(logits.device, nbytes, workspace, True, stream=stream)
    at = ints.data_ptr()
    _call("moe_route", stream, (logits,), logits.data_ptr(), T, E, k, 1 if renormalize else 0, at, weights.data_ptr(),
          at + 12 * R, at + 4 * R, at + 8 * R, ws_ptr, ws_bytes)
    return Routing(experts, weights, offsets, positions, tokens)


def _scratch(like, nbytes, stream):
    """A workspace for one call, which needs no initialisation.  Allocated on
    the stream that uses it, so that its memory is handed out again in order."""
    torch = _torch_module
    if stream is None:
        return like.new_empty((nbytes,), dtype=torch.uint8)
    with torch.cuda.stream(stream):
        return like.new_empty((nbytes,), dtype=torch.uint8)


def moe_route_grad(dweights, logits, experts, weights, renormalize=True, out=None, stream=None):
    """dlogits [T, E] from the gradient of moe_route's weights."""
    torch = _torch_module
    _need(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    _need(experts, torch.int32, "experts", 2)
    k = experts.shape[1]
    _need_shape(experts, torch.int32, (T, k), "experts")
    _need_shape(weights, torch.float32, (T, k), "weights")
    _need_shape(dweights, torch.float32, (T, k), "dweights")
    out = _out(out, torch.float32, (T, E), logits, stream)
    _call("moe_route_grad", stream, (logits, dweights, experts, weights, out), dweights.data_ptr(), logits.data_ptr(),
          experts.data_ptr(), weights.data_ptr(), T, E, k, 1 if renormalize else 0, out.data_ptr())
    return out


def moe_dispatch(X, positions, out=None, stream=None):
    """Rows in the grouped order: out[positions[t, j]] = X[t] for X [T, H]
    (BF16 or FP32, H a multiple of 8); out [T*k, H]."""
    torch = _torch_module
    code = _row_code(X, "X")
    T, H = X.shape
    _need(positions, torch.int32, "positions", 2)
    k = positions.shape[1]
    _need_shape(positions, torch.int32, (T, k), "positions")
    out = _out(out, X.dtype, (T * k, H), X, stream)
    _call("moe_dispatch", stream, (X, positions, out), X.data_ptr(), positions.data_ptr(), T, k, H, code,
          out.data_ptr())
    return out


def _grouped_rows(rows, positions, weights):
    """(dtype code, T, k, H) of rows [T*k, H], positions and weights [T, k]."""
    torch = _torch_module
    code = _row_code(rows, "rows")
    R, H = rows.shape
    _need(positions, torch.int32, "positions", 2)
    T, k = positions.shape
    if R != T * k:
        raise ValueError(f"rows has {R} rows, positions {T} x {k}")
    if weights is not None:
        _need_shape(weights, torch.float32, (T, k), "weights")
    return code, T, k, H


def moe_combine(rows, positions, weights=None, out=None, stream=None):
    """Rows back in token order: out[t] = sum_j weights[t, j] *
    rows[positions[t, j]] (FP32 sum, one rounding to the rows' dtype).  Without
    weights this is the gradient of moe_dispatch."""
    code, T, k, H = _grouped_rows(rows, positions, weights)
    out = _out(out, rows.dtype, (T, H), rows, stream)
    _call("moe_combine", stream, (rows, positions, weights, out), rows.data_ptr(), positions.data_ptr(),
          weights.data_ptr() if weights is not None else None, T, k, H, code, out.data_ptr())
    return out


def moe_combine_grad(dout, rows, positions, weights, stream=None):
    """Gradients of the weighted moe_combine: (drows [T*k, H] in the rows'
    dtype, dweights [T, k] FP32)."""
    code, T, k, H = _grouped_rows(rows, positions, weights)
    _need_shape(dout, rows.dtype, (T, H), "dout")
    drows, dweights = _new(rows.shape, rows.dtype, rows, stream), _new((T, k), weights.dtype, rows, stream)
    _call("moe_combine_grad", stream, (dout, rows, positions, weights), dout.data_ptr(), rows.data_ptr(),
          positions.data_ptr(), weights.data_ptr(), T, k, H, code, drows.data_ptr(), dweights.data_ptr())
    return drows, dweights


def quantize_int8(X, positions=None, stream=None):
    """Codes and scales of the rows of X [T, K] (BF16 or FP32, K a multiple of
    16): (q int8 [T, K], scale FP32 [T]).  With positions [T, k] each token's
    codes go to its k rows of the grouped order: q [T*k, K], scale [T*k]."""
    torch = _torch_module
    code = _row_code(X, "X")
    T, K = X.shape
    k, at = 1, None
    if positions is not None:
        _need(positions, torch.int32, "positions", 2)
        k, at = positions.shape[1], positions.data_ptr()
        _need_shape(positions, torch.int32, (T, k), "positions")
    q = _new((T * k, K), torch.int8, X, stream)
    scale = _new((T * k,), torch.float32, X, stream)
    _call("quantize_int8", stream, (X, positions), X.data_ptr(), code, T, K, at, k, q.data_ptr(), scale.data_ptr())
    return q, scale


def _int8_operands(Xq, x_scale, Wq, w_scale, wdim, M, gated, out_dtype, out, stream):
    torch = _torch_module
    _need(Xq, torch.int8, "Xq", 2)
    _need(Wq, torch.int8, "Wq", wdim)
    _need(x_scale, torch.float32, "x_scale", 1)
    _need(w_scale, torch.float32, "w_scale", wdim - 1)
    T, K = Xq.shape
    N = Wq.shape[-2]
    if Wq.shape[-1] != K or x_scale.shape[0] != T or w_scale.shape != Wq.shape[:-1]:
        raise ValueError(f"shape mismatch: Xq {tuple(Xq.shape)}, x_scale {tuple(x_scale.shape)}, "
                         f"Wq {tuple(Wq.shape)}, w_scale {tuple(w_scale.shape)}")
    code = BF16 if out_dtype is None else _dtype_code(out_dtype)
    out = _out(out, _torch_dtype(code), (T if M is None else M, N // 2 if gated else N), Xq, stream)
    return T, N, K, code, out


def grouped_gemm_int8(Xq, x_scale, Wq, w_scale, group_offsets, gated=False, rows=None, out_dtype=None, out=None,
                      stream=None):
    """Y[t] = x_scale[t] * w_scale[e(t)] * (Xq[t] Wq[e(t)]^T) for int8 codes Xq
    [M, K], Wq [E, N, K] and FP32 scales [M], [E, N]: an exact integer sum,
    scaled in FP32 and rounded once to out_dtype (bf16 by default).  gated:
    the N = 2I columns are gate and up halves, and Y [M, I] = silu(gate) * up.
    rows (int32 [M], moe_route's tokens): row t of the product is row rows[t]
    of Xq [T, K] and x_scale [T], T*K < 2^31 - 4096."""
    torch = _torch_module
    E = _offsets(group_offsets)
    M = at = None
    if rows is not None:
        _need(rows, torch.int32, "rows", 1)
        M, at = rows.numel(), rows.data_ptr()
    T, N, K, code, out = _int8_operands(Xq, x_scale, Wq, w_scale, 3, M, gated, out_dtype, out, stream)
    if Wq.shape[0] != E:
        raise ValueError(f"shape mismatch: Wq {tuple(Wq.shape)}, E={E}")
    _call("grouped_gemm_int8", stream, (Xq, x_scale, Wq, w_scale, group_offsets, rows, out), Xq.data_ptr(),
          x_scale.data_ptr(), Wq.data_ptr(), w_scale.data_ptr(), group_offsets.data_ptr(), at, T, E,
          T if M is None else M, N, K, 1 if gated else 0, code, out.data_ptr())
    return out


def gemm_int8(Xq, x_scale, Wq, w_scale, gated=False, out_dtype=None, out=None, stream=None):
    """The one-group case of grouped_gemm_int8: Wq [N, K], w_scale [N]."""
    M, N, K, code, out = _int8_operands(Xq, x_scale, Wq, w_scale, 2, None, gated, out_dtype, out, stream)
    _call("gemm_int8", stream, (Xq, x_scale, Wq, w_scale, out), Xq.data_ptr(), x_scale.data_ptr(), Wq.data_ptr(),
          w_scale.data_ptr(), M, N, K, 1 if gated else 0, code, out.data_ptr())
    return out


def moe_ffn_int8(X, logits, W1q, w1_scale, W2q, w2_scale, k, renormalize=True, out=None, workspace=None, stream=None):
    """A gated feed-forward block of E experts in one call: moe_route on logits
    [T, E], quantize_int8 of X [T, H] (BF16), the gated product of its rows in
    the grouped order with W1q [E, 2I, H] (FP32 result), quantize_int8 of it, the product
    with W2q [E, H, I] (BF16) and moe_combine: [T, H] BF16.  `workspace`: a
    device tensor of at least ffn_workspace_size bytes, or None for one
    allocated for this call."""
    torch = _torch_module
    _need(X, torch.bfloat16, "X", 2)
    T, H = X.shape
    _need(logits, torch.float32, "logits", 2)
    E = logits.shape[1]
    _need_shape(logits, torch.float32, (T, E), "logits")
    _need(W1q, torch.int8, "W1q", 3)
    N = W1q.shape[1]
    I = N // 2
    _need_shape(W1q, torch.int8, (E, 2 * I, H), "W1q")
    _need_shape(w1_scale, torch.float32, (E, N), "w1_scale")
    _need_shape(W2q, torch.int8, (E, H, I), "W2q")
    _need_shape(w2_scale, torch.float32, (E, H), "w2_scale")
    out = _out(out, torch.bfloat16, (T, H), X, stream)
    if workspace is None:
        workspace = _scratch(X, ffn_workspace_size(T, E, k, H, I), stream)
    else:
        _need_span(workspace)
    _call("moe_ffn_int8", stream, (X, logits, W1q, w1_scale, W2q, w2_scale, out, workspace), X.data_ptr(),
          logits.data_ptr(), W1q.data_ptr(), w1_scale.data_ptr(), W2q.data_ptr(), w2_scale.data_ptr(), T, E, int(k), H,
          I, 1 if renormalize else 0, out.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


def ffn_workspace_size(T: int, E: int, k: int, H: int, I: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.moe_ffn_int8_workspace_size(T, E, k, H, I, ctypes.byref(n)), "moe_ffn_int8_workspace_size")
    return n.value


# ---- selection by scores ---------------------------------------------------------

class Scoring(NamedTuple):
    """How moe_route_scores chooses and weighs: `score` "sigmoid" or "softmax";
    `bias` FP32 [E] (added to the score for the choice alone) or None; the E
    experts in `groups` groups of neighbours, of which the top_groups take part
    whose largest value (best=1), or the sum of their two largest (best=2), is
    largest; weights renormalised over the chosen or not, times `scale`."""
    score: str = "sigmoid"
    bias: "torch.Tensor | None" = None
    groups: int = 1
    top_groups: int = 1
    best: int = 2
    renormalize: bool = True
    scale: float = 1.0


_SCORES = {"softmax": 0, "sigmoid": 1}


def _scoring(c, E):
    """The C structure of a Scoring (its bias is not kept alive by it)."""
    if c.score not in _SCORES:
        raise ValueError(f"unknown score {c.score!r}: sigmoid or softmax")
    at = None
    if c.bias is not None:
        _need_shape(c.bias, _torch_module.float32, (E,), "bias")
        at = c.bias.data_ptr()
    return ScoringStruct(_SCORES[c.score], c.groups, c.top_groups, c.best, 1 if c.renormalize else 0, c.scale, at)


def moe_route_scores(logits, k, scoring=Scoring(), workspace=None, stream=None):
    """moe_route on scores of the logits [T, E] (FP32), chosen and weighted as
    the Scoring says: a Routing.  Choices are those of 64-bit values, ties to
    the lowest index.  A masked (-inf) logit, or a bias of -inf, is chosen last
    and gets weight 0."""
    torch = _torch_module
    _need(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    k = int(k)
    c = _scoring(scoring, E)
    nbytes = route_workspace_size(T, E, k)
    R = T * k
    weights = _new((T, k), torch.float32, logits, stream)
    ints = _new((3 * R + E + 1,), torch.int32, logits, stream)   # one allocation, as in moe_route
    experts, positions = ints.as_strided((T, k), (k, 1)), ints.as_strided((T, k), (k, 1), R)
    tokens, offsets = ints.as_strided((R,), (1,), 2 * R), ints.as_strided((E + 1,), (1,), 3 * R)
    ws_ptr, ws_bytes = None, 0
    if nbytes and workspace is None:
        scratch = _scratch(logits, nbytes, stream)
        ws_ptr, ws_bytes = scratch.data_ptr(), nbytes
    elif nbytes:
        ws_ptr, ws_bytes = _workspace(logits.device, nbytes, workspace, True, stream=stream)
    at = ints.data_ptr()
    _call("moe_route_scores", stream, (logits, scoring.bias), logits.data_ptr(), T, E, k, c, at, weights.data_ptr(),
          at + 12 * R, at + 4 * R, at + 8 * R, ws_ptr, ws_bytes)
    return Routing(experts, weights, offsets, positions, tokens)


def moe_route_scores_grad(dweights, logits, experts, weights, scoring=Scoring(), out=None, stream=None):
    """dlogits [T, E] from the gradient of moe_route_scores' weights."""
    torch = _torch_module
    _need(logits, torch.float32, "logits", 2)
    T, E = logits.shape
    _need(experts, torch.int32, "experts", 2)
    k = experts.shape[1]
    _need_shape(experts, torch.int32, (T, k), "experts")
    _need_shape(weights, torch.float32, (T, k), "weights")
    _need_shape(dweights, torch.float32, (T, k), "dweights")
    c = _scoring(scoring._replace(bias=None), E)
    out = _out(out, torch.float32, (T, E), logits, stream)
    _call("moe_route_scores_grad", stream, (logits, dweights, experts, weights, out), dweights.data_ptr(),
          logits.data_ptr(), experts.data_ptr(), weights.data_ptr(), T, E, k, c, out.data_ptr())
    return out


# ---- microscaled 4-bit floating point ---------------------------------------------

def mxfp4_scales(scales):
    """Scale bytes [.., rows, K/32], one after another in each row as other
    programs store them, in the layout that the 4-bit products read:
    [ceil(K/256), .., rows, 8]."""
    torch = _torch_module
    if scales.dtype != torch.uint8 or scales.dim() < 2:
        raise TypeError("scales must be uint8 with at least two dimensions")
    blocks = -(-scales.shape[-1] // 8)
    padded = torch.nn.functional.pad(scales, (0, 8 * blocks - scales.shape[-1]))
    return padded.unflatten(-1, (blocks, 8)).movedim(-2, 0).contiguous()


def quantize_mxfp4(X, stream=None):
    """Codes and scales of the rows of X [T, K] (BF16 or FP32, K a multiple of
    32): (codes uint8 [T, K/2], scales uint8 [ceil(K/256), T, 8])."""
    torch = _torch_module
    code = _row_code(X, "X")
    T, K = X.shape
    codes = _new((T, K // 2), torch.uint8, X, stream)
    scales = _new((-(-K // 256), T, 8), torch.uint8, X, stream)
    _call("quantize_mxfp4", stream, (X,), X.data_ptr(), code, T, K, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def _mx_operand(codes, scales, dims, what):
    """K of codes [.., K/2] whose scales have their shape."""
    torch = _torch_module
    _need(codes, torch.uint8, what, dims)
    _need(scales, torch.uint8, f"{what}'s scales", dims + 1)
    K = 2 * codes.shape[-1]
    if scales.shape != (-(-K // 256), *codes.shape[:-1], 8):
        raise ValueError(f"{what} is {tuple(codes.shape)}, its scales {tuple(scales.shape)}")
    return K


def dequantize_mxfp4(codes, scales, dtype=None, out=None, stream=None):
    """The values [T, K] that quantize_mxfp4's codes and scales stand for, BF16
    (default) or FP32."""
    K = _mx_operand(codes, scales, 2, "codes")
    code = BF16 if dtype is None else _dtype_code(dtype)
    T = codes.shape[0]
    out = _out(out, _torch_dtype(code), (T, K), codes, stream)
    _call("dequantize_mxfp4", stream, (codes, scales, out), codes.data_ptr(), scales.data_ptr(), T, K, code, out.data_ptr())
    return out


def _mx_operands(Xq, x_scale, Wq, w_scale, wdim, M, gated, out_dtype, out, stream):
    K, Kw = _mx_operand(Xq, x_scale, 2, "Xq"), _mx_operand(Wq, w_scale, wdim, "Wq")
    if K != Kw:
        raise ValueError(f"shape mismatch: Xq {tuple(Xq.shape)}, Wq {tuple(Wq.shape)}")
    T, N = Xq.shape[0], Wq.shape[-2]
    code = BF16 if out_dtype is None else _dtype_code(out_dtype)
    out = _out(out, _torch_dtype(code), (T if M is None else M, N // 2 if gated else N), Xq, stream)
    return T, N, K, code, out


def grouped_gemm_mxfp4(Xq, x_scale, Wq, w_scale, group_offsets, gated=False, rows=None, out_dtype=None, out=None,
                       stream=None):
    """Y[t] = x[t] w[e(t)]^T for 4-bit codes Xq [M, K/2], Wq [E, N, K/2] with
    scales [ceil(K/256), M, 8], [ceil(K/256), E, N, 8]: FP32 accumulation of
    exact products, rounded once to out_dtype (bf16 by default).  gated and
    rows as for grouped_gemm_int8; with rows, Xq [T, K/2], T*K/2 < 2^31 - 4096."""
    torch = _torch_module
    E = _offsets(group_offsets)
    M = at = None
    if rows is not None:
        _need(rows, torch.int32, "rows", 1)
        M, at = rows.numel(), rows.data_ptr()
    T, N, K, code, out = _mx_operands(Xq, x_scale, Wq, w_scale, 3, M, gated, out_dtype, out, stream)
    if Wq.shape[0] != E:
        raise ValueError(f"shape mismatch: Wq {tuple(Wq.shape)}, E={E}")
    _call("grouped_gemm_mxfp4", stream, (Xq, x_scale, Wq, w_scale, group_offsets, rows, out), Xq.data_ptr(),
          x_scale.data_ptr(), Wq.data_ptr(), w_scale.data_ptr(), group_offsets.data_ptr(), at, T, E,
          T if M is None else M, N, K, 1 if gated else 0, code, out.data_ptr())
    return out


def gemm_mxfp4(Xq, x_scale, Wq, w_scale, gated=False, out_dtype=None, out=None, stream=None):
    """The one-group case of grouped_gemm_mxfp4: Wq [N, K/2], w_scale
    [ceil(K/256), N, 8]."""
    M, N, K, code, out = _mx_operands(Xq, x_scale, Wq, w_scale, 2, None, gated, out_dtype, out, stream)
    _call("gemm_mxfp4", stream, (Xq, x_scale, Wq, w_scale, out), Xq.data_ptr(), x_scale.data_ptr(), Wq.data_ptr(),
          w_scale.data_ptr(), M, N, K, 1 if gated else 0, code, out.data_ptr())
    return out


def moe_ffn_mxfp4(X, logits, W1q, w1_scale, W2q, w2_scale, k, scoring=None, out=None, workspace=None, stream=None):
    """moe_ffn_int8's block on 4-bit weights in one call: the selection (by
    `scoring`, or moe_route's with renormalised weights), quantize_mxfp4 of X
    [T, H] (BF16), the gated product with W1q [E, 2I, H/2] (FP32 result),
    quantize_mxfp4 of it, the product with W2q [E, H, I/2] (BF16) and
    moe_combine: [T, H] BF16.  `workspace`: a device tensor of at least
    ffn_mxfp4_workspace_size bytes, or None for one allocated for this call."""
    torch = _torch_module
    _need(X, torch.bfloat16, "X", 2)
    T, H = X.shape
    _need(logits, torch.float32, "logits", 2)
    E = logits.shape[1]
    _need_shape(logits, torch.float32, (T, E), "logits")
    K1, I = _mx_operand(W1q, w1_scale, 3, "W1q"), _mx_operand(W2q, w2_scale, 3, "W2q")
    if K1 != H or W1q.shape[:2] != (E, 2 * I) or W2q.shape[:2] != (E, H):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W1q {tuple(W1q.shape)}, W2q {tuple(W2q.shape)}, E={E}")
    c = None if scoring is None else _scoring(scoring, E)
    out = _out(out, torch.bfloat16, (T, H), X, stream)
    if workspace is None:
        workspace = _scratch(X, ffn_mxfp4_workspace_size(T, E, k, H, I), stream)
    else:
        _need_span(workspace)
    _call("moe_ffn_mxfp4", stream, (X, logits, W1q, w1_scale, W2q, w2_scale, out, workspace,
                                    None if scoring is None else scoring.bias), X.data_ptr(), logits.data_ptr(),
          W1q.data_ptr(), w1_scale.data_ptr(), W2q.data_ptr(), w2_scale.data_ptr(), T, E, int(k), H, I, c, out.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def ffn_mxfp4_workspace_size(T: int, E: int, k: int, H: int, I: int) -> int:
    n = ctypes.c_size_t()
    _check(lib.moe_ffn_mxfp4_workspace_size(T, E, k, H, I, ctypes.byref(n)), "moe_ffn_mxfp4_workspace_size")
    return n.value


# ---- the gated activation kept in 8 bits -------------------------------------------

KEPT_BLOCK = 128   # columns of a half that share a scale


def _gate_rows(positions, weights, R):
    torch = _torch_module
    _need(positions, torch.int32, "positions", 2)
    T, k = positions.shape
    if R != T * k:
        raise ValueError(f"{R} rows, positions {T} x {k}")
    _need_shape(weights, torch.float32, (T, k), "weights")
    return T, k


def moe_gate_int8(GU, positions, weights, stream=None):
    """The gated activation of grouped rows with their weights, and what its
    gradient needs: GU [T*k, 2I] BF16 (gate, then up) to (h [T*k, I] BF16 =
    weight * silu(gate) * up, codes int8 [T*k, 2I], scale FP32 [T*k,
    2*ceil(I/128)], one for each 128 columns of a half).  positions and weights
    [T, k] as moe_route gives them; a row of weight 0 gives zeros whatever it
    holds.  The rows that the next product makes of h are added by moe_combine
    without weights."""
    torch = _torch_module
    _need(GU, torch.bfloat16, "GU", 2)
    R, N = GU.shape
    if N % 2:
        raise ValueError("GU needs a gate and an up half")
    T, k = _gate_rows(positions, weights, R)
    I = N // 2
    h = _new((R, I), torch.bfloat16, GU, stream)
    codes = _new((R, N), torch.int8, GU, stream)
    scale = _new((R, 2 * -(-I // KEPT_BLOCK)), torch.float32, GU, stream)
    _call("moe_gate_int8", stream, (GU, positions, weights), GU.data_ptr(), positions.data_ptr(), weights.data_ptr(), T, k, I,
          h.data_ptr(), codes.data_ptr(), scale.data_ptr())
    return h, codes, scale


def moe_gate_int8_grad(dh, codes, scale, positions, weights, stream=None):
    """From dh [T*k, I] BF16 and what moe_gate_int8 kept: (dGU [T*k, 2I] BF16,
    h [T*k, I] BF16 again, dweights [T, k] FP32), the gradients at the values
    that the codes stand for."""
    torch = _torch_module
    _need(dh, torch.bfloat16, "dh", 2)
    R, I = dh.shape
    T, k = _gate_rows(positions, weights, R)
    _need_shape(codes, torch.int8, (R, 2 * I), "codes")
    _need_shape(scale, torch.float32, (R, 2 * -(-I // KEPT_BLOCK)), "scale")
    dGU = _new((R, 2 * I), torch.bfloat16, dh, stream)
    h = _new((R, I), torch.bfloat16, dh, stream)
    dweights = _new((T, k), torch.float32, dh, stream)
    _call("moe_gate_int8_grad", stream, (dh, codes, scale, positions, weights), dh.data_ptr(), codes.data_ptr(),
          scale.data_ptr(), positions.data_ptr(), weights.data_ptr(), T, k, I, dGU.data_ptr(), h.data_ptr(),
          dweights.data_ptr())
    return dGU, h, dweights


if os.environ.get("DRGG_NO_ROUTES", "0") in ("", "0"):
    load_default_routes()
