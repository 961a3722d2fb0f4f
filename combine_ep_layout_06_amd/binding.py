"""ctypes binding of libep_mi355x.so (include/ep.h) for torch tensors.

Argument marshalling only: each function checks dtypes, devices, sizes and contiguity, then
passes ``data_ptr()`` values and torch's current HIP stream to the C entry point of the same
name. Under ``record()`` the C calls are captured into a CallList instead, whose ``replay()``
re-issues them without the Python-side checks (for loops that refill the same buffers). What a
call with ``stream=`` allocates (outputs not passed in, a workspace) is memory of that stream. Every
step of the computation runs in the library's gfx950 kernels; there is no other code path. If
the library is missing the functions raise instead of computing anything.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from .build import LIB

EP_OK, EP_ERR_INVALID, EP_ERR_ALIGN, EP_ERR_UNSUPPORTED, EP_ERR_HIP = 0, -1, -2, -3, -4
EP_STATS_LEN = 4
EP_MAX_EXPERTS = 1024
EP_MAX_TOPK = 256
EP_FP8_BLOCK = 128
EP_MAX_RANKS = 64
EP_MOE_MAX_PAIRS = 2048

#: every entry point the header declares
EXPORTED = ("ep_layout", "ep_dispatch", "ep_dispatch_fp8", "ep_layout_dispatch",
            "ep_layout_dispatch_fp8", "ep_combine", "ep_rank_layout", "ep_dispatch_ranks",
            "ep_dispatch_ranks_fp8", "ep_rank_layout_dispatch", "ep_rank_layout_dispatch_fp8",
            "ep_dispatch_expand", "ep_dispatch_expand_fp8", "ep_layout_dispatch_expand",
            "ep_layout_dispatch_expand_fp8",
            "ep_combine_ranks", "ep_combine_reduce", "ep_layout_packed", "ep_dispatch_packed",
            "ep_dispatch_packed_fp8", "ep_layout_dispatch_packed", "ep_layout_dispatch_packed_fp8",
            "ep_combine_packed", "ep_check_e4m3_conversion", "ep_last_launches",
            "ep_layout_workspace_bytes", "ep_layout_dispatch_ws", "ep_layout_dispatch_fp8_ws",
            "ep_layout_dispatch_noalloc", "ep_expert_gemm_fp8", "ep_expert_gemm_fp8_packed",
            "ep_expert_swiglu_fp8", "ep_expert_swiglu_fp8_packed", "ep_moe_layer",
            "ep_moe_layer_fp8", "ep_moe_layer_workspace_bytes", "ep_expert_gemm",
            "ep_expert_gemm_packed", "ep_expert_swiglu", "ep_expert_swiglu_packed",
            "ep_expert_gemm_dgrad", "ep_expert_gemm_dgrad_packed", "ep_expert_swiglu_dgrad",
            "ep_expert_swiglu_dgrad_packed", "ep_expert_gemm_wgrad", "ep_expert_gemm_wgrad_packed",
            "ep_expert_gemm_wgrad_f32", "ep_expert_gemm_wgrad_f32_packed", "ep_combine_grad",
            "ep_combine_grad_packed", "ep_linear", "ep_linear_grad",
            "ep_linear_grad_workspace_bytes", "ep_error_string", "ep_last_error", "ep_version")

#: activations of ep_linear by name (EP_ACT_* of the header)
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


class EpShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("C", ctypes.c_int32), ("R", ctypes.c_int32)]


class EpLaunchRecord(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p),
                ("grid_x", ctypes.c_uint32), ("grid_y", ctypes.c_uint32),
                ("grid_z", ctypes.c_uint32), ("block_x", ctypes.c_uint32),
                ("block_y", ctypes.c_uint32), ("block_z", ctypes.c_uint32),
                ("dynamic_lds_bytes", ctypes.c_uint32), ("static_lds_bytes", ctypes.c_uint32),
                ("vgprs", ctypes.c_int32), ("private_bytes", ctypes.c_uint32),
                ("max_threads_per_block", ctypes.c_int32)]


class EpError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str):
        super().__init__(f"{fn} failed with {code}: {detail}")
        self.code = code


_lib = None
_int_places = {}       # per C call: where its 32-bit integers are among its arguments after the shape


def library_path() -> str:
    return os.environ.get("EP_MI355X_LIB", LIB)


def load_library():
    """Load the HIP library once. Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m combine_ep_layout_06_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(path)
        vp, sp = ctypes.c_void_p, ctypes.POINTER(EpShape)
        L.ep_layout.argtypes = [sp] + [vp] * 7 + [vp]
        L.ep_dispatch.argtypes = [sp, vp, vp, vp, vp, vp]
        L.ep_dispatch_fp8.argtypes = [sp, vp, vp, vp, vp, vp, vp]
        L.ep_combine.argtypes = [sp, vp, vp, vp, vp, vp, vp]
        L.ep_layout_dispatch.argtypes = [sp] + [vp] * 10
        L.ep_layout_dispatch_fp8.argtypes = [sp] + [vp] * 11
        L.ep_rank_layout.argtypes = [sp, vp, vp, vp, vp]
        L.ep_dispatch_ranks.argtypes = [sp, vp, vp, vp, vp]
        L.ep_dispatch_ranks_fp8.argtypes = [sp, vp, vp, vp, vp, vp]
        L.ep_rank_layout_dispatch.argtypes = [sp] + [vp] * 6
        L.ep_rank_layout_dispatch_fp8.argtypes = [sp] + [vp] * 7
        L.ep_dispatch_expand.argtypes = [sp] + [vp] * 6
        L.ep_dispatch_expand_fp8.argtypes = [sp] + [vp] * 8
        L.ep_layout_dispatch_expand.argtypes = [sp] + [vp] * 11
        L.ep_layout_dispatch_expand_fp8.argtypes = [sp] + [vp] * 13
        L.ep_combine_ranks.argtypes = [sp] + [vp] * 7
        L.ep_combine_reduce.argtypes = [sp] + [vp] * 4
        i32 = ctypes.c_int32
        L.ep_layout_packed.argtypes = [sp, i32] + [vp] * 8
        L.ep_dispatch_packed.argtypes = [sp, i32] + [vp] * 6
        L.ep_dispatch_packed_fp8.argtypes = [sp, i32] + [vp] * 7
        L.ep_combine_packed.argtypes = [sp, i32] + [vp] * 7
        L.ep_layout_dispatch_packed.argtypes = [sp, i32, i32] + [vp] * 10
        L.ep_layout_dispatch_packed_fp8.argtypes = [sp, i32, i32] + [vp] * 11
        L.ep_check_e4m3_conversion.argtypes = [ctypes.c_uint32, ctypes.c_uint32, vp, vp, vp]
        L.ep_last_launches.argtypes = [ctypes.POINTER(EpLaunchRecord), ctypes.c_int]
        L.ep_layout_dispatch_ws.argtypes = [sp] + [vp] * 10 + [ctypes.c_size_t, vp]
        L.ep_layout_dispatch_fp8_ws.argtypes = [sp] + [vp] * 11 + [ctypes.c_size_t, vp]
        L.ep_layout_dispatch_noalloc.argtypes = [sp] + [vp] * 10
        L.ep_expert_gemm_fp8.argtypes = [sp, i32] + [vp] * 7
        L.ep_expert_gemm_fp8_packed.argtypes = [sp, i32, i32] + [vp] * 8
        L.ep_expert_swiglu_fp8.argtypes = [sp, i32] + [vp] * 8
        L.ep_expert_swiglu_fp8_packed.argtypes = [sp, i32, i32] + [vp] * 9
        L.ep_moe_layer.argtypes = [sp, i32] + [vp] * 7 + [ctypes.c_size_t, vp]
        L.ep_moe_layer_fp8.argtypes = [sp, i32] + [vp] * 9 + [ctypes.c_size_t, vp]
        L.ep_moe_layer_workspace_bytes.argtypes = [sp, i32]
        L.ep_moe_layer_workspace_bytes.restype = ctypes.c_size_t
        L.ep_expert_gemm.argtypes = [sp, i32] + [vp] * 5
        L.ep_expert_gemm_packed.argtypes = [sp, i32, i32] + [vp] * 6
        L.ep_expert_swiglu.argtypes = [sp, i32] + [vp] * 6
        L.ep_expert_swiglu_packed.argtypes = [sp, i32, i32] + [vp] * 7
        L.ep_expert_gemm_dgrad.argtypes = [sp, i32] + [vp] * 5
        L.ep_expert_gemm_dgrad_packed.argtypes = [sp, i32, i32] + [vp] * 6
        L.ep_expert_swiglu_dgrad.argtypes = [sp, i32] + [vp] * 6
        L.ep_expert_swiglu_dgrad_packed.argtypes = [sp, i32, i32] + [vp] * 7
        L.ep_expert_gemm_wgrad.argtypes = [sp, i32] + [vp] * 5
        L.ep_expert_gemm_wgrad_packed.argtypes = [sp, i32, i32] + [vp] * 6
        L.ep_expert_gemm_wgrad_f32.argtypes = [sp, i32, i32] + [vp] * 5
        L.ep_expert_gemm_wgrad_f32_packed.argtypes = [sp, i32, i32, i32] + [vp] * 6
        L.ep_combine_grad.argtypes = [sp] + [vp] * 8
        L.ep_combine_grad_packed.argtypes = [sp, i32] + [vp] * 9
        L.ep_linear.argtypes = [sp, i32, i32] + [vp] * 7
        L.ep_linear_grad.argtypes = [sp, i32, i32] + [vp] * 8 + [ctypes.c_size_t, vp]
        L.ep_linear_grad_workspace_bytes.argtypes = [sp, i32, i32]
        for fn in EXPORTED:
            if fn.startswith("ep_") and fn not in ("ep_error_string", "ep_last_error",
                                                   "ep_version", "ep_layout_workspace_bytes",
                                                   "ep_moe_layer_workspace_bytes",
                                                   "ep_linear_grad_workspace_bytes"):
                getattr(L, fn).restype = ctypes.c_int
        for fn in EXPORTED:
            types = getattr(L, fn).argtypes or ()
            _int_places[fn] = [i for i, t in enumerate(types[1:]) if t is i32]
        L.ep_layout_workspace_bytes.argtypes = [sp]
        L.ep_layout_workspace_bytes.restype = ctypes.c_size_t
        L.ep_linear_grad_workspace_bytes.restype = ctypes.c_size_t
        L.ep_error_string.argtypes = [ctypes.c_int]
        L.ep_error_string.restype = ctypes.c_char_p
        L.ep_last_error.argtypes = []
        L.ep_last_error.restype = ctypes.c_char_p
        L.ep_version.argtypes = []
        L.ep_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def ep_version() -> str:
    return load_library().ep_version().decode()


def ep_error_string(code: int) -> str:
    return load_library().ep_error_string(code).decode()


def _check(fn: str, rc: int):
    if rc != EP_OK:
        raise EpError(fn, rc, load_library().ep_last_error().decode())


_shapes: dict = {}


def _shape(T, H, E, K, C, R) -> EpShape:
    # one EpShape per distinct shape (the C calls only read it)
    key = (T, H, E, K, C, R)
    sh = _shapes.get(key)
    if sh is None:
        if len(_shapes) >= 4096:
            _shapes.clear()
        values = [int(v) for v in key]
        if any(v != ctypes.c_int32(v).value for v in values):      # a field would keep its low half
            raise ValueError(f"a shape's T, H, E, K, C, R must fit 32 bits: {values}")
        sh = _shapes[key] = EpShape(*values)
    return sh


# torch's current HIP stream of the current device as a raw handle, without building a Stream
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


class CallList:
    """Entry-point calls captured by `record`: the same C calls with the same device pointers,
    re-issued by `replay` with none of the wrappers' checks or allocations. It holds references
    to every tensor the calls use, so the buffers live as long as the list."""

    def __init__(self):
        self.calls = []      # (C function, name, shape, pointer and int arguments, stream)
        self._tensors = []
        self.device = None   # the device of the recorded tensors

    def __len__(self):
        return len(self.calls)

    def replay(self, stream=None):
        """Issue the recorded calls in order, each on the stream it was recorded with if one was
        given then, else on ``stream`` (default: torch's current stream)."""
        if not self.calls:
            return
        _require_current("replay", self.device)
        s = _stream(stream)
        for fn, name, sh, args, st in self.calls:
            rc = fn(ctypes.byref(sh), *args, s if st is None else st)
            if rc != EP_OK:
                _check(name, rc)


_recording = threading.local()


@contextlib.contextmanager
def record():
    """Inside the block, the entry-point functions validate their arguments and allocate any
    missing outputs as usual, but the C calls are captured instead of issued. Yields the
    CallList; its ``replay()`` then launches the same kernels on the same buffers, which is
    all a serving loop needs when each step refills the same input tensors."""
    prev = getattr(_recording, "calls", None)
    cl = CallList()
    _recording.calls = cl
    try:
        yield cl
    finally:
        _recording.calls = prev


def _require_current(name: str, dev):
    """The library launches on the current HIP device, so the tensors must live there (device
    pointers of another GPU, or host pointers, would be read by the kernels)."""
    if dev is not None and dev.type == "cuda" and dev.index == torch.cuda.current_device():
        return
    try:
        cur = f"cuda:{torch.cuda.current_device()}"
    except RuntimeError:
        cur = "none (no GPU)"
    raise ValueError(f"{name}: the tensors are on {dev}, but the library launches on the current "
                     f"HIP device ({cur}); move them there or call under torch.cuda.device()")


def _fits32(name: str, value: int):
    if not -2147483648 <= value <= 2147483647:     # ctypes would pass its low half
        raise ValueError(f"{name}: a size of {value} does not fit 32 bits")


def _call(name: str, sh: EpShape, *args, stream=None):
    """Issue (or record) one C call; tensor arguments are passed as their data pointers."""
    fn = getattr(load_library(), name)
    for i in _int_places[name]:
        if not -2147483648 <= args[i] <= 2147483647:
            _fits32(name, args[i])
    cargs = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    dev = next((a.device for a in args if isinstance(a, torch.Tensor)), None)
    cl = getattr(_recording, "calls", None)
    if cl is not None:
        if cl.calls and dev != cl.device:
            raise ValueError(f"{name}: a recorded list holds calls on one device only "
                             f"({cl.device}, not {dev})")
        cl.device = dev
        cl._tensors.extend([a for a in args if isinstance(a, torch.Tensor)])
        cl.calls.append((fn, name, sh, tuple(cargs),
                         None if stream is None else stream.cuda_stream))
        return
    _require_current(name, dev)
    rc = fn(ctypes.byref(sh), *cargs, _stream(stream))
    if rc != EP_OK:
        _check(name, rc)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, numel: int, device):
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() != numel:
        _reject(t, name, dtype, numel, device)


def _reject(t: torch.Tensor, name: str, dtype: torch.dtype, numel: int, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")


def _bf16(t: torch.Tensor) -> torch.dtype:
    # bf16 rows may be passed as torch.bfloat16 or as their int16/uint16 bit patterns
    return t.dtype if t.dtype in (torch.bfloat16, torch.int16, torch.uint16) else torch.bfloat16


def _new(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """An output that the caller did not pass in. For a call on another stream it is memory of that
    stream (a block of the current one may have work of its last owner pending, which the call would
    not wait for), not reused before the current stream's work at its release is done either."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def ep_layout(topk_idx: torch.Tensor, E: int, C: int, R: int, *, slot=None, expert_count=None,
              expert_offset=None, rank_count=None, rank_offset=None, stats=None, stream=None):
    """Routing layout. ``topk_idx`` int32 [T, K] on the GPU. Returns a dict of the outputs
    (``slot`` [T, K], ``expert_count`` [E], ``expert_offset`` [E], ``rank_count`` [R],
    ``rank_offset`` [R], ``stats`` [4] = kept, dropped, unrouted, invalid); any of them may be
    passed in preallocated."""
    dev = topk_idx.device
    T, K = topk_idx.shape
    mk = lambda n: _new(n, torch.int32, dev, stream)
    slot = mk((T, K)) if slot is None else slot
    expert_count = mk(E) if expert_count is None else expert_count
    expert_offset = mk(E) if expert_offset is None else expert_offset
    rank_count = mk(R) if rank_count is None else rank_count
    rank_offset = mk(R) if rank_offset is None else rank_offset
    stats = mk(EP_STATS_LEN) if stats is None else stats
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    for name, t, n in (("expert_count", expert_count, E), ("expert_offset", expert_offset, E),
                       ("rank_count", rank_count, R), ("rank_offset", rank_offset, R),
                       ("stats", stats, EP_STATS_LEN)):
        _need(t, name, torch.int32, n, dev)
    sh = _shape(T, 1, E, K, C, R)
    _call("ep_layout", sh, topk_idx, slot, expert_count, expert_offset, rank_count, rank_offset,
          stats, stream=stream)
    return dict(slot=slot, expert_count=expert_count, expert_offset=expert_offset,
                rank_count=rank_count, rank_offset=rank_offset, stats=stats)


def _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                    rank_offset, stats):
    mk = lambda n: _new(n, torch.int32, dev, stream)
    out = dict(slot=mk((T, K)) if slot is None else slot,
               expert_count=mk(E) if expert_count is None else expert_count,
               expert_offset=mk(E) if expert_offset is None else expert_offset,
               rank_count=mk(R) if rank_count is None else rank_count,
               rank_offset=mk(R) if rank_offset is None else rank_offset,
               stats=mk(EP_STATS_LEN) if stats is None else stats)
    _need(out["slot"], "slot", torch.int32, T * K, dev)
    for name, n in (("expert_count", E), ("expert_offset", E), ("rank_count", R),
                    ("rank_offset", R), ("stats", EP_STATS_LEN)):
        _need(out[name], name, torch.int32, n, dev)
    return out


def _layout_ts(lay):
    return [lay[k] for k in ("slot", "expert_count", "expert_offset", "rank_count",
                             "rank_offset", "stats")]


def ep_layout_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, recv: torch.Tensor, E: int,
                       C: int, R: int, *, slot=None, expert_count=None, expert_offset=None,
                       rank_count=None, rank_offset=None, stats=None, stream=None):
    """ep_layout + bf16 dispatch in one launch. Returns the layout dict (as ep_layout);
    ``recv`` [E, C, H] is written in place."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv, "recv", _bf16(recv), E * C * H, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch", sh, x, topk_idx, *_layout_ts(lay), recv, stream=stream)
    return lay


def layout_workspace_bytes(T: int, K: int, E: int) -> int:
    """Bytes of workspace the _ws calls need for T tokens, top-K, E experts."""
    return int(load_library().ep_layout_workspace_bytes(ctypes.byref(_shape(T, 1, E, K, 1, 1))))


def _own_workspace(nbytes: int, dev, stream):
    """A workspace that lives for one call, as memory of the stream the call runs on: the allocator
    then hands it out and takes it back in that stream's order. (A block of another stream may have
    work of its last owner pending there, which the call would not wait for.)"""
    on = contextlib.nullcontext() if stream is None or dev.type != "cuda" else torch.cuda.stream(stream)
    with on:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)


def _workspace(workspace, T, K, E, dev, stream):
    need = layout_workspace_bytes(T, K, E)
    if workspace is None:
        workspace = _own_workspace(need, dev, stream)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous tensor on the batch's device")
    return workspace, workspace.numel() * workspace.element_size()


def ep_layout_dispatch_ws(x: torch.Tensor, topk_idx: torch.Tensor, recv: torch.Tensor, E: int,
                          C: int, R: int, *, workspace=None, slot=None, expert_count=None,
                          expert_offset=None, rank_count=None, rank_offset=None, stats=None,
                          stream=None):
    """ep_layout_dispatch in two launches through a workspace (chunk histograms): the same
    outputs, faster on large batches. ``workspace``: a device tensor of at least
    layout_workspace_bytes(T, K, E) bytes (allocated here if not given)."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv, "recv", _bf16(recv), E * C * H, dev)
    ws, nbytes = _workspace(workspace, T, K, E, dev, stream)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_ws", sh, x, topk_idx, *_layout_ts(lay), recv, ws, nbytes,
          stream=stream)
    return lay


def ep_layout_dispatch_noalloc(x: torch.Tensor, topk_idx: torch.Tensor, recv: torch.Tensor,
                               E: int, C: int, R: int, *, slot=None, expert_count=None,
                               expert_offset=None, rank_count=None, rank_offset=None, stats=None,
                               stream=None):
    """ep_layout_dispatch_ws with the library's static scratch as the workspace (no workspace
    argument; the C call allocates nothing). Pass every output to allocate nothing here
    either."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv, "recv", _bf16(recv), E * C * H, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_noalloc", sh, x, topk_idx, *_layout_ts(lay), recv, stream=stream)
    return lay


def ep_layout_dispatch_fp8_ws(x: torch.Tensor, topk_idx: torch.Tensor, recv_q: torch.Tensor,
                              recv_scale: torch.Tensor, E: int, C: int, R: int, *,
                              workspace=None, slot=None, expert_count=None, expert_offset=None,
                              rank_count=None, rank_offset=None, stats=None, stream=None):
    """ep_layout_dispatch_fp8 in two launches through a workspace (see ep_layout_dispatch_ws)."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv_q, "recv_q", recv_q.dtype if recv_q.dtype in (torch.uint8, torch.float8_e4m3fn)
          else torch.uint8, E * C * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, E * C * (H // EP_FP8_BLOCK), dev)
    ws, nbytes = _workspace(workspace, T, K, E, dev, stream)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_fp8_ws", sh, x, topk_idx, *_layout_ts(lay), recv_q, recv_scale,
          ws, nbytes, stream=stream)
    return lay


def ep_layout_dispatch_fp8(x: torch.Tensor, topk_idx: torch.Tensor, recv_q: torch.Tensor,
                           recv_scale: torch.Tensor, E: int, C: int, R: int, *, slot=None,
                           expert_count=None, expert_offset=None, rank_count=None,
                           rank_offset=None, stats=None, stream=None):
    """ep_layout + FP8 dispatch in one launch. Returns the layout dict; ``recv_q`` and
    ``recv_scale`` are written in place."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv_q, "recv_q", recv_q.dtype if recv_q.dtype in (torch.uint8, torch.float8_e4m3fn)
          else torch.uint8, E * C * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, E * C * (H // EP_FP8_BLOCK), dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_fp8", sh, x, topk_idx, *_layout_ts(lay), recv_q, recv_scale,
          stream=stream)
    return lay


def ep_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor, recv: torch.Tensor,
                C: int, *, stream=None):
    """bf16 dispatch: ``x`` [T, H] bf16 -> ``recv`` [E, C, H] bf16 (written in place)."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    E = recv.numel() // (C * H)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(recv, "recv", _bf16(recv), E * C * H, dev)
    sh = _shape(T, H, E, K, C, 1)
    _call("ep_dispatch", sh, x, topk_idx, slot, recv, stream=stream)
    return recv


def ep_dispatch_fp8(x: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                    recv_q: torch.Tensor, recv_scale: torch.Tensor, C: int, *, stream=None):
    """FP8 dispatch: ``x`` [T, H] bf16 -> ``recv_q`` [E, C, H] uint8 (OCP E4M3 codes) and
    ``recv_scale`` [E, C, H/128] float32 (written in place)."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    E = recv_q.numel() // (C * H)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(recv_q, "recv_q", recv_q.dtype if recv_q.dtype in (torch.uint8, torch.float8_e4m3fn)
          else torch.uint8, E * C * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, E * C * (H // EP_FP8_BLOCK), dev)
    sh = _shape(T, H, E, K, C, 1)
    _call("ep_dispatch_fp8", sh, x, topk_idx, slot, recv_q, recv_scale, stream=stream)
    return recv_q, recv_scale


def ep_combine(y: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
               topk_w: torch.Tensor, C: int, *, out=None, stream=None):
    """Combine: ``y`` [E, C, H] bf16 -> ``out`` [T, H] bf16."""
    dev = y.device
    T, K = topk_idx.shape
    H = y.shape[-1]
    E = y.numel() // (C * H)
    out = _new((T, H), _bf16(y), dev, stream) if out is None else out
    _need(y, "y", _bf16(y), E * C * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(topk_w, "topk_w", torch.float32, T * K, dev)
    _need(out, "out", _bf16(out), T * H, dev)
    sh = _shape(T, H, E, K, C, 1)
    _call("ep_combine", sh, y, topk_idx, slot, topk_w, out, stream=stream)
    return out


# ------------------------------------------------------------------------------------------
# two-stage, rank-deduplicated path (stage buffers are [R, T, ...])
# ------------------------------------------------------------------------------------------

def ep_rank_layout(topk_idx: torch.Tensor, E: int, R: int, *, rank_slot=None, rank_tokens=None,
                   stream=None):
    """Which virtual ranks each token goes to: ``rank_slot`` int32 [T, R] (position among the
    rank's tokens, -1 if not sent) and ``rank_tokens`` int32 [R]."""
    dev = topk_idx.device
    T, K = topk_idx.shape
    rank_slot = _new((T, R), torch.int32, dev, stream) if rank_slot is None else rank_slot
    rank_tokens = (_new(R, torch.int32, dev, stream) if rank_tokens is None
                   else rank_tokens)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(rank_tokens, "rank_tokens", torch.int32, R, dev)
    sh = _shape(T, 1, E, K, 1, R)
    _call("ep_rank_layout", sh, topk_idx, rank_slot, rank_tokens, stream=stream)
    return dict(rank_slot=rank_slot, rank_tokens=rank_tokens)


def ep_dispatch_ranks(x: torch.Tensor, rank_slot: torch.Tensor, stage: torch.Tensor, *,
                      stream=None):
    """Stage 1 of dispatch: ``x`` [T, H] bf16 -> ``stage`` [R, T, H] bf16 (in place)."""
    dev = x.device
    T, H = x.shape
    R = rank_slot.shape[1]
    _need(x, "x", _bf16(x), T * H, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(stage, "stage", _bf16(stage), R * T * H, dev)
    sh = _shape(T, H, R, 1, 1, R)
    _call("ep_dispatch_ranks", sh, x, rank_slot, stage, stream=stream)
    return stage


def ep_dispatch_ranks_fp8(x: torch.Tensor, rank_slot: torch.Tensor, stage_q: torch.Tensor,
                          stage_scale: torch.Tensor, *, stream=None):
    """FP8 stage 1: ``stage_q`` [R, T, H] uint8 and ``stage_scale`` [R, T, H/128] float32."""
    dev = x.device
    T, H = x.shape
    R = rank_slot.shape[1]
    _need(x, "x", _bf16(x), T * H, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(stage_q, "stage_q", torch.uint8, R * T * H, dev)
    _need(stage_scale, "stage_scale", torch.float32, R * T * (H // EP_FP8_BLOCK), dev)
    sh = _shape(T, H, R, 1, 1, R)
    _call("ep_dispatch_ranks_fp8", sh, x, rank_slot, stage_q, stage_scale, stream=stream)
    return stage_q, stage_scale


def ep_rank_layout_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, E: int, R: int, *,
                            stage=None, rank_slot=None, rank_tokens=None, stream=None):
    """ep_rank_layout and ep_dispatch_ranks in one launch: ``x`` [T, H] bf16 -> ``stage``
    [R, T, H] bf16 (rows of tokens a rank does not receive untouched), ``rank_slot`` [T, R],
    ``rank_tokens`` [R]."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    stage = _new((R, T, H), _bf16(x), dev, stream) if stage is None else stage
    rank_slot = _new((T, R), torch.int32, dev, stream) if rank_slot is None else rank_slot
    rank_tokens = (_new(R, torch.int32, dev, stream) if rank_tokens is None
                   else rank_tokens)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(rank_tokens, "rank_tokens", torch.int32, R, dev)
    _need(stage, "stage", _bf16(stage), R * T * H, dev)
    sh = _shape(T, H, E, K, 1, R)
    _call("ep_rank_layout_dispatch", sh, x, topk_idx, rank_slot, rank_tokens, stage, stream=stream)
    return dict(stage=stage, rank_slot=rank_slot, rank_tokens=rank_tokens)


def ep_rank_layout_dispatch_fp8(x: torch.Tensor, topk_idx: torch.Tensor, E: int, R: int, *,
                                stage_q=None, stage_scale=None, rank_slot=None,
                                rank_tokens=None, stream=None):
    """ep_rank_layout and ep_dispatch_ranks_fp8 in one launch: ``stage_q`` [R, T, H] uint8,
    ``stage_scale`` [R, T, H/128] float32, ``rank_slot`` [T, R], ``rank_tokens`` [R]."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    NB = H // EP_FP8_BLOCK
    stage_q = _new((R, T, H), torch.uint8, dev, stream) if stage_q is None else stage_q
    stage_scale = (_new((R, T, NB), torch.float32, dev, stream)
                   if stage_scale is None else stage_scale)
    rank_slot = _new((T, R), torch.int32, dev, stream) if rank_slot is None else rank_slot
    rank_tokens = (_new(R, torch.int32, dev, stream) if rank_tokens is None
                   else rank_tokens)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(rank_tokens, "rank_tokens", torch.int32, R, dev)
    _need(stage_q, "stage_q", torch.uint8, R * T * H, dev)
    _need(stage_scale, "stage_scale", torch.float32, R * T * NB, dev)
    sh = _shape(T, H, E, K, 1, R)
    _call("ep_rank_layout_dispatch_fp8", sh, x, topk_idx, rank_slot, rank_tokens, stage_q,
          stage_scale, stream=stream)
    return dict(stage_q=stage_q, stage_scale=stage_scale, rank_slot=rank_slot,
                rank_tokens=rank_tokens)


def ep_dispatch_expand(stage: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                       rank_slot: torch.Tensor, recv: torch.Tensor, C: int, *, stream=None):
    """Stage 2 of dispatch: ``stage`` [R, T, H] -> ``recv`` [E, C, H] bf16 (in place)."""
    dev = stage.device
    R, T, H = stage.shape
    K = topk_idx.shape[1]
    E = recv.numel() // (C * H)
    _need(stage, "stage", _bf16(stage), R * T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(recv, "recv", _bf16(recv), E * C * H, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_dispatch_expand", sh, stage, topk_idx, slot, rank_slot, recv, stream=stream)
    return recv


def ep_layout_dispatch_expand(stage: torch.Tensor, topk_idx: torch.Tensor,
                              rank_slot: torch.Tensor, recv: torch.Tensor, E: int, C: int, *,
                              slot=None, expert_count=None, expert_offset=None, rank_count=None,
                              rank_offset=None, stats=None, stream=None):
    """ep_layout + stage 2 of dispatch in one launch: ``stage`` [R, T, H] -> ``recv`` [E, C, H]
    bf16 (in place). Returns the layout dict (as ep_layout)."""
    dev = stage.device
    R, T, H = stage.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(stage, "stage", _bf16(stage), R * T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(recv, "recv", _bf16(recv), E * C * H, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_expand", sh, stage, topk_idx, rank_slot, *_layout_ts(lay), recv,
          stream=stream)
    return lay


def ep_layout_dispatch_expand_fp8(stage_q: torch.Tensor, stage_scale: torch.Tensor,
                                  topk_idx: torch.Tensor, rank_slot: torch.Tensor,
                                  recv_q: torch.Tensor, recv_scale: torch.Tensor, E: int, C: int,
                                  *, slot=None, expert_count=None, expert_offset=None,
                                  rank_count=None, rank_offset=None, stats=None, stream=None):
    """ep_layout + FP8 stage 2 in one launch: codes and scales of the staged rows -> ``recv_q``
    [E, C, H] and ``recv_scale`` [E, C, H/128] (in place). Returns the layout dict."""
    dev = stage_q.device
    R, T, H = stage_q.shape
    K = topk_idx.shape[1]
    lay = _layout_outputs(dev, stream, T, K, E, R, slot, expert_count, expert_offset, rank_count,
                          rank_offset, stats)
    _need(stage_q, "stage_q", stage_q.dtype if stage_q.dtype in (torch.uint8, torch.float8_e4m3fn)
          else torch.uint8, R * T * H, dev)
    _need(stage_scale, "stage_scale", torch.float32, R * T * (H // EP_FP8_BLOCK), dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(recv_q, "recv_q", recv_q.dtype if recv_q.dtype in (torch.uint8, torch.float8_e4m3fn)
          else torch.uint8, E * C * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, E * C * (H // EP_FP8_BLOCK), dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_expand_fp8", sh, stage_q, stage_scale, topk_idx, rank_slot,
          *_layout_ts(lay), recv_q, recv_scale, stream=stream)
    return lay


def ep_dispatch_expand_fp8(stage_q: torch.Tensor, stage_scale: torch.Tensor,
                           topk_idx: torch.Tensor, slot: torch.Tensor, rank_slot: torch.Tensor,
                           recv_q: torch.Tensor, recv_scale: torch.Tensor, C: int, *,
                           stream=None):
    """FP8 stage 2: codes and scales of the staged rows -> ``recv_q`` [E, C, H] and
    ``recv_scale`` [E, C, H/128] (in place)."""
    dev = stage_q.device
    R, T, H = stage_q.shape
    K = topk_idx.shape[1]
    E = recv_q.numel() // (C * H)
    NB = H // EP_FP8_BLOCK
    _need(stage_q, "stage_q", torch.uint8, R * T * H, dev)
    _need(stage_scale, "stage_scale", torch.float32, R * T * NB, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(recv_q, "recv_q", torch.uint8, E * C * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, E * C * NB, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_dispatch_expand_fp8", sh, stage_q, stage_scale, topk_idx, slot, rank_slot, recv_q,
          recv_scale, stream=stream)
    return recv_q, recv_scale


def ep_combine_ranks(y: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                     rank_slot: torch.Tensor, topk_w: torch.Tensor, C: int, *, part=None,
                     stream=None):
    """Stage 1 of combine: ``y`` [E, C, H] bf16 -> per-rank partial rows ``part`` [R, T, H]."""
    dev = y.device
    T, K = topk_idx.shape
    R = rank_slot.shape[1]
    H = y.shape[-1]
    E = y.numel() // (C * H)
    part = _new((R, T, H), _bf16(y), dev, stream) if part is None else part
    _need(y, "y", _bf16(y), E * C * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(topk_w, "topk_w", torch.float32, T * K, dev)
    _need(part, "part", _bf16(part), R * T * H, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_combine_ranks", sh, y, topk_idx, slot, rank_slot, topk_w, part, stream=stream)
    return part


def ep_combine_reduce(part: torch.Tensor, rank_slot: torch.Tensor, K: int, *, out=None,
                      stream=None):
    """Stage 2 of combine: ``part`` [R, T, H] -> ``out`` [T, H] bf16. K (the top-k of the
    routing) bounds the ranks a token reaches."""
    dev = part.device
    R, T, H = part.shape
    out = _new((T, H), _bf16(part), dev, stream) if out is None else out
    _need(part, "part", _bf16(part), R * T * H, dev)
    _need(rank_slot, "rank_slot", torch.int32, T * R, dev)
    _need(out, "out", _bf16(out), T * H, dev)
    sh = _shape(T, H, R, K, 1, R)
    _call("ep_combine_reduce", sh, part, rank_slot, out, stream=stream)
    return out


# ------------------------------------------------------------------------------------------
# packed, aligned receive layout (buffers are [rows, ...])
# ------------------------------------------------------------------------------------------

def packed_rows_bound(T: int, K: int, E: int, C: int, alignment: int) -> int:
    """Rows that always suffice for a packed buffer: every kept pair plus each expert's padding."""
    return min(T * K, E * C) + E * (alignment - 1)


def ep_layout_packed(topk_idx: torch.Tensor, E: int, C: int, R: int, alignment: int, *,
                     slot=None, expert_count=None, packed_offset=None, rank_count=None,
                     rank_offset=None, stats=None, stream=None):
    """Layout with packed offsets: returns ``slot``, ``expert_count``, ``packed_offset``
    [E + 1] (offset of each expert's rows, then the rows needed), ``rank_count``,
    ``rank_offset`` (padded rows per rank) and ``stats``."""
    dev = topk_idx.device
    T, K = topk_idx.shape
    mk = lambda n: _new(n, torch.int32, dev, stream)
    slot = mk((T, K)) if slot is None else slot
    expert_count = mk(E) if expert_count is None else expert_count
    packed_offset = mk(E + 1) if packed_offset is None else packed_offset
    rank_count = mk(R) if rank_count is None else rank_count
    rank_offset = mk(R) if rank_offset is None else rank_offset
    stats = mk(EP_STATS_LEN) if stats is None else stats
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    for name, t, n in (("expert_count", expert_count, E), ("packed_offset", packed_offset, E + 1),
                       ("rank_count", rank_count, R), ("rank_offset", rank_offset, R),
                       ("stats", stats, EP_STATS_LEN)):
        _need(t, name, torch.int32, n, dev)
    sh = _shape(T, 1, E, K, C, R)
    _call("ep_layout_packed", sh, int(alignment), topk_idx, slot, expert_count, packed_offset,
          rank_count, rank_offset, stats, stream=stream)
    return dict(slot=slot, expert_count=expert_count, packed_offset=packed_offset,
                rank_count=rank_count, rank_offset=rank_offset, stats=stats)


def ep_dispatch_packed(x: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                       packed_offset: torch.Tensor, recv: torch.Tensor, E: int, C: int, *,
                       stream=None):
    """bf16 dispatch into the packed ``recv`` [rows, H] (in place)."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    rows = recv.shape[0]
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(packed_offset, "packed_offset", torch.int32, E + 1, dev)
    _need(recv, "recv", _bf16(recv), rows * H, dev)
    sh = _shape(T, H, E, K, C, 1)
    _call("ep_dispatch_packed", sh, int(rows), x, topk_idx, slot, packed_offset, recv,
          stream=stream)
    return recv


def ep_dispatch_packed_fp8(x: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                           packed_offset: torch.Tensor, recv_q: torch.Tensor,
                           recv_scale: torch.Tensor, E: int, C: int, *, stream=None):
    """FP8 dispatch into the packed ``recv_q`` [rows, H] and ``recv_scale`` [rows, H/128]."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    rows = recv_q.shape[0]
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(packed_offset, "packed_offset", torch.int32, E + 1, dev)
    _need(recv_q, "recv_q", torch.uint8, rows * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, rows * (H // EP_FP8_BLOCK), dev)
    sh = _shape(T, H, E, K, C, 1)
    _call("ep_dispatch_packed_fp8", sh, int(rows), x, topk_idx, slot, packed_offset, recv_q,
          recv_scale, stream=stream)
    return recv_q, recv_scale


def _packed_layout_outputs(dev, stream, T, K, E, R, slot, expert_count, packed_offset, rank_count,
                           rank_offset, stats):
    mk = lambda n: _new(n, torch.int32, dev, stream)
    out = dict(slot=mk((T, K)) if slot is None else slot,
               expert_count=mk(E) if expert_count is None else expert_count,
               packed_offset=mk(E + 1) if packed_offset is None else packed_offset,
               rank_count=mk(R) if rank_count is None else rank_count,
               rank_offset=mk(R) if rank_offset is None else rank_offset,
               stats=mk(EP_STATS_LEN) if stats is None else stats)
    _need(out["slot"], "slot", torch.int32, T * K, dev)
    for name, n in (("expert_count", E), ("packed_offset", E + 1), ("rank_count", R),
                    ("rank_offset", R), ("stats", EP_STATS_LEN)):
        _need(out[name], name, torch.int32, n, dev)
    return out


def ep_layout_dispatch_packed(x: torch.Tensor, topk_idx: torch.Tensor, recv: torch.Tensor, E: int,
                              C: int, R: int, alignment: int, *, slot=None, expert_count=None,
                              packed_offset=None, rank_count=None, rank_offset=None, stats=None,
                              stream=None):
    """ep_layout_packed and ep_dispatch_packed in one launch: the packed layout's outputs (a
    dict as ep_layout_packed returns) and ``recv`` [rows, H] bf16 filled in place."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    rows = recv.shape[0]
    o = _packed_layout_outputs(dev, stream, T, K, E, R, slot, expert_count, packed_offset, rank_count,
                               rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv, "recv", _bf16(recv), rows * H, dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_packed", sh, int(alignment), int(rows), x, topk_idx, o["slot"],
          o["expert_count"], o["packed_offset"], o["rank_count"], o["rank_offset"], o["stats"],
          recv, stream=stream)
    return o


def ep_layout_dispatch_packed_fp8(x: torch.Tensor, topk_idx: torch.Tensor, recv_q: torch.Tensor,
                                  recv_scale: torch.Tensor, E: int, C: int, R: int,
                                  alignment: int, *, slot=None, expert_count=None,
                                  packed_offset=None, rank_count=None, rank_offset=None,
                                  stats=None, stream=None):
    """ep_layout_packed and ep_dispatch_packed_fp8 in one launch: the packed layout's outputs,
    ``recv_q`` [rows, H] and ``recv_scale`` [rows, H/128] filled in place."""
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    rows = recv_q.shape[0]
    o = _packed_layout_outputs(dev, stream, T, K, E, R, slot, expert_count, packed_offset, rank_count,
                               rank_offset, stats)
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(recv_q, "recv_q", torch.uint8, rows * H, dev)
    _need(recv_scale, "recv_scale", torch.float32, rows * (H // EP_FP8_BLOCK), dev)
    sh = _shape(T, H, E, K, C, R)
    _call("ep_layout_dispatch_packed_fp8", sh, int(alignment), int(rows), x, topk_idx, o["slot"],
          o["expert_count"], o["packed_offset"], o["rank_count"], o["rank_offset"], o["stats"],
          recv_q, recv_scale, stream=stream)
    return o


def ep_combine_packed(y: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                      packed_offset: torch.Tensor, topk_w: torch.Tensor, E: int, C: int, *,
                      out=None, stream=None):
    """Combine from the packed ``y`` [rows, H] -> ``out`` [T, H] bf16."""
    dev = y.device
    T, K = topk_idx.shape
    rows, H = y.shape
    out = _new((T, H), _bf16(y), dev, stream) if out is None else out
    _need(y, "y", _bf16(y), rows * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(slot, "slot", torch.int32, T * K, dev)
    _need(packed_offset, "packed_offset", torch.int32, E + 1, dev)
    _need(topk_w, "topk_w", torch.float32, T * K, dev)
    _need(out, "out", _bf16(out), T * H, dev)
    sh = _shape(T, H, E, K, C, 1)
    _call("ep_combine_packed", sh, int(rows), y, topk_idx, slot, packed_offset, topk_w, out,
          stream=stream)
    return out


# ------------------------------------------------------------------------------------------
# the experts between dispatch and combine
# ------------------------------------------------------------------------------------------

def _e4m3(t: torch.Tensor) -> torch.dtype:
    # FP8 codes may be passed as torch.float8_e4m3fn or as their uint8 bit patterns
    return t.dtype if t.dtype in (torch.uint8, torch.float8_e4m3fn) else torch.uint8


def _product_args(q, scale, expert_count, w_q, w_scale, lead):
    """Checks of the rows and weights of an experts' product; returns (E, n, H)."""
    if w_q.dim() != 3 or q.dim() != lead + 1:
        raise ValueError(f"expected rows with {lead + 1} dimensions and w_q [E, N, H], got "
                         f"{tuple(q.shape)} and {tuple(w_q.shape)}")
    E, n, H = w_q.shape
    if q.shape[-1] != H or (lead == 2 and q.shape[0] != E):
        raise ValueError(f"rows {tuple(q.shape)} do not fit the weights {tuple(w_q.shape)}")
    dev = q.device
    nb = H // EP_FP8_BLOCK
    _need(q, "recv_q", _e4m3(q), q.numel(), dev)
    _need(scale, "recv_scale", torch.float32, q.numel() // H * nb if H else 0, dev)
    _need(expert_count, "expert_count", torch.int32, E, dev)
    _need(w_q, "w_q", _e4m3(w_q), E * n * H, dev)
    _need(w_scale, "w_scale", torch.float32, E * -(-n // EP_FP8_BLOCK) * nb, dev)
    return E, n, H


def ep_expert_gemm_fp8(recv_q: torch.Tensor, recv_scale: torch.Tensor,
                       expert_count: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor,
                       pairs: int, *, y=None, stream=None):
    """The experts' product on a padded receive buffer: ``recv_q`` [E, C, H] E4M3 codes and
    ``recv_scale`` [E, C, H/128] float32 (as ep_dispatch_fp8 writes them), the first
    ``expert_count[e]`` rows of each expert; weights ``w_q`` [E, N, H] codes and ``w_scale``
    [E, ceil(N/128), H/128] -> ``y`` [E, C, N] bf16. Rows that hold no pair are neither read nor
    written. ``pairs``: T * K, the pairs the layout placed (chooses the grid, never the result;
    0: nothing is computed)."""
    E, N, H = _product_args(recv_q, recv_scale, expert_count, w_q, w_scale, 2)
    C, dev = recv_q.shape[1], recv_q.device
    y = _new((E, C, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", _bf16(y), E * C * N, dev)
    sh = _shape(pairs, H, E, 1, C, 1)
    _call("ep_expert_gemm_fp8", sh, N, recv_q, recv_scale, expert_count, w_q, w_scale, y,
          stream=stream)
    return y


def ep_expert_gemm_fp8_packed(recv_q: torch.Tensor, recv_scale: torch.Tensor,
                              expert_count: torch.Tensor, packed_offset: torch.Tensor,
                              w_q: torch.Tensor, w_scale: torch.Tensor, pairs: int, *, y=None,
                              stream=None):
    """ep_expert_gemm_fp8 on a packed buffer: ``recv_q`` [rows, H], ``recv_scale`` [rows, H/128],
    expert e's rows from ``packed_offset[e]`` on -> ``y`` [rows, N] bf16."""
    E, N, H = _product_args(recv_q, recv_scale, expert_count, w_q, w_scale, 1)
    rows, dev = recv_q.shape[0], recv_q.device
    _need(packed_offset, "packed_offset", torch.int32, E + 1, dev)
    y = _new((rows, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", _bf16(y), rows * N, dev)
    sh = _shape(pairs, H, E, 1, 1, 1)
    _call("ep_expert_gemm_fp8_packed", sh, rows, N, recv_q, recv_scale, expert_count,
          packed_offset, w_q, w_scale, y, stream=stream)
    return y


def ep_expert_swiglu_fp8(recv_q: torch.Tensor, recv_scale: torch.Tensor,
                         expert_count: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor,
                         pairs: int, *, h_q=None, h_scale=None, stream=None):
    """The gate and up products, SwiGLU and the FP8 cast on a padded receive buffer: the rows of
    ep_expert_gemm_fp8, ``w_q`` [E, 2I, H] (the I gate rows, then the I up rows) and ``w_scale``
    [E, 2I/128, H/128] -> ``h_q`` [E, C, I] E4M3 codes and ``h_scale`` [E, C, I/128] float32,
    which ep_expert_gemm_fp8 takes as its rows."""
    E, n, H = _product_args(recv_q, recv_scale, expert_count, w_q, w_scale, 2)
    if n % 2:
        raise ValueError(f"w_q: expected an even number of rows (gate, then up), got {n}")
    C, I, dev = recv_q.shape[1], n // 2, recv_q.device
    h_q = _new((E, C, I), recv_q.dtype, dev, stream) if h_q is None else h_q
    h_scale = (_new((E, C, I // EP_FP8_BLOCK), torch.float32, dev, stream)
               if h_scale is None else h_scale)
    _need(h_q, "h_q", _e4m3(h_q), E * C * I, dev)
    _need(h_scale, "h_scale", torch.float32, E * C * (I // EP_FP8_BLOCK), dev)
    sh = _shape(pairs, H, E, 1, C, 1)
    _call("ep_expert_swiglu_fp8", sh, I, recv_q, recv_scale, expert_count, w_q, w_scale, h_q,
          h_scale, stream=stream)
    return h_q, h_scale


def ep_expert_swiglu_fp8_packed(recv_q: torch.Tensor, recv_scale: torch.Tensor,
                                expert_count: torch.Tensor, packed_offset: torch.Tensor,
                                w_q: torch.Tensor, w_scale: torch.Tensor, pairs: int, *,
                                h_q=None, h_scale=None, stream=None):
    """ep_expert_swiglu_fp8 on a packed buffer: ``recv_q`` [rows, H] -> ``h_q`` [rows, I] and
    ``h_scale`` [rows, I/128]."""
    E, n, H = _product_args(recv_q, recv_scale, expert_count, w_q, w_scale, 1)
    if n % 2:
        raise ValueError(f"w_q: expected an even number of rows (gate, then up), got {n}")
    rows, I, dev = recv_q.shape[0], n // 2, recv_q.device
    _need(packed_offset, "packed_offset", torch.int32, E + 1, dev)
    h_q = _new((rows, I), recv_q.dtype, dev, stream) if h_q is None else h_q
    h_scale = (_new((rows, I // EP_FP8_BLOCK), torch.float32, dev, stream)
               if h_scale is None else h_scale)
    _need(h_q, "h_q", _e4m3(h_q), rows * I, dev)
    _need(h_scale, "h_scale", torch.float32, rows * (I // EP_FP8_BLOCK), dev)
    sh = _shape(pairs, H, E, 1, 1, 1)
    _call("ep_expert_swiglu_fp8_packed", sh, rows, I, recv_q, recv_scale, expert_count,
          packed_offset, w_q, w_scale, h_q, h_scale, stream=stream)
    return h_q, h_scale

def moe_layer_workspace_bytes(T: int, K: int, H: int, I: int) -> int:
    """Bytes of workspace a whole-layer call needs for T tokens of H channels, top-K,
    intermediate size I."""
    return int(load_library().ep_moe_layer_workspace_bytes(
        ctypes.byref(_shape(T, H, 1, K, 1, 1)), I))


def _moe_layer(name, x, topk_idx, topk_w, w13, w2, dtype, out, workspace, stream):
    """Checks shared by the whole-layer calls; returns what both C calls take."""
    if x.dim() != 2 or topk_idx.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError(f"{name}: expected x [T, H], topk_idx [T, K], w13 [E, 2I, H] and "
                         f"w2 [E, H, I]")
    dev = x.device
    (T, H), K, (E, n, _), I = x.shape, topk_idx.shape[1], w13.shape, w2.shape[2]
    if n != 2 * I or topk_idx.shape[0] != T or w13.shape[2] != H or w2.shape[:2] != (E, H):
        raise ValueError(f"{name}: x {tuple(x.shape)}, topk_idx {tuple(topk_idx.shape)}, w13 "
                         f"{tuple(w13.shape)} and w2 {tuple(w2.shape)} do not fit together")
    _need(x, "x", _bf16(x), T * H, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * K, dev)
    _need(topk_w, "topk_w", torch.float32, T * K, dev)
    _need(w13, "w13", dtype(w13), E * n * H, dev)
    _need(w2, "w2", dtype(w2), E * H * I, dev)
    out = _new((T, H), _bf16(x), dev, stream) if out is None else out
    _need(out, "out", _bf16(out), T * H, dev)
    if workspace is None:
        # more pairs are refused below, whatever the workspace
        need = moe_layer_workspace_bytes(T, K, H, I) if T * K <= EP_MOE_MAX_PAIRS else 0
        workspace = _own_workspace(need, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous tensor on the tokens' device")
    return (_shape(T, H, E, K, 1, 1), I, out, workspace,
            workspace.numel() * workspace.element_size())


def ep_moe_layer(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                 w13: torch.Tensor, w2: torch.Tensor, *, out=None, workspace=None, stream=None):
    """A whole MoE layer for a few tokens (T * K <= EP_MOE_MAX_PAIRS), in two or three launches:
    ``out[t] = sum_j topk_w[t, j] * W2[e_j] (silu(Wg[e_j] x[t]) * (Wu[e_j] x[t]))`` with bf16
    weights ``w13`` [E, 2I, H] (gate rows, then up rows) and ``w2`` [E, H, I]; ``x`` and ``out``
    [T, H] bf16. Pairs whose id is not a valid expert add nothing. ``workspace``: a device tensor
    of at least moe_layer_workspace_bytes(T, K, H, I) bytes (allocated here if not given)."""
    sh, I, out, ws, nbytes = _moe_layer("ep_moe_layer", x, topk_idx, topk_w, w13, w2, _bf16, out,
                                        workspace, stream)
    _call("ep_moe_layer", sh, I, x, topk_idx, topk_w, w13, w2, out, ws, nbytes, stream=stream)
    return out


def ep_moe_layer_fp8(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                     w13_q: torch.Tensor, w13_scale: torch.Tensor, w2_q: torch.Tensor,
                     w2_scale: torch.Tensor, *, out=None, workspace=None, stream=None):
    """ep_moe_layer with FP8 weights: E4M3 codes ``w13_q`` [E, 2I, H] and ``w2_q`` [E, H, I] and
    one float32 scale per 128 x 128 block, ``w13_scale`` [E, 2I/128, H/128] and ``w2_scale``
    [E, H/128, I/128]. Activations stay bf16."""
    sh, I, out, ws, nbytes = _moe_layer("ep_moe_layer_fp8", x, topk_idx, topk_w, w13_q, w2_q,
                                        _e4m3, out, workspace, stream)
    E, (H, dev) = sh.E, (sh.H, x.device)
    _need(w13_scale, "w13_scale", torch.float32,
          E * (2 * I // EP_FP8_BLOCK) * (H // EP_FP8_BLOCK), dev)
    _need(w2_scale, "w2_scale", torch.float32, E * (H // EP_FP8_BLOCK) * (I // EP_FP8_BLOCK), dev)
    _call("ep_moe_layer_fp8", sh, I, x, topk_idx, topk_w, w13_q, w13_scale, w2_q, w2_scale, out,
          ws, nbytes, stream=stream)
    return out


# ------------------------------------------------------------------------------------------
# the experts in bf16, forward and backward
# ------------------------------------------------------------------------------------------

_BF16_TYPES = (torch.bfloat16, torch.int16, torch.uint16)


def _rows(t: torch.Tensor, name: str, shape: tuple, device):
    """Checks that `t` holds bf16 values in this shape."""
    if t.shape != shape or t.dtype not in _BF16_TYPES or t.device != device or not t.is_contiguous():
        if t.shape != shape:
            raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")
        _need(t, name, _bf16(t), t.numel(), device)


def _weights3(w: torch.Tensor, name: str):
    if w.dim() != 3:
        raise ValueError(f"{name}: expected three dimensions, [E, rows, columns], got {tuple(w.shape)}")
    return w.shape


def _experts(expert_count: torch.Tensor) -> int:
    if expert_count.dim() != 1:
        raise ValueError(f"expert_count: expected [E], got {tuple(expert_count.shape)}")
    return expert_count.shape[0]


def _expert_rows(x: torch.Tensor, name: str, E: int, expert_count: torch.Tensor, packed_offset):
    """The leading sizes of a receive buffer, [E, C, width] or with `packed_offset` [rows, width],
    with the counts and offsets checked; and the buffer's device."""
    shape, dev = x.shape, x.device
    if len(shape) != (3 if packed_offset is None else 2):
        raise ValueError(f"{name}: expected {'[E, C, width]' if packed_offset is None else '[rows, width]'}"
                         f", got {tuple(shape)}")
    if packed_offset is None and shape[0] != E:
        raise ValueError(f"{name}: {shape[0]} experts' rows for {E} experts")
    _need(expert_count, "expert_count", torch.int32, E, dev)
    if packed_offset is not None:
        _need(packed_offset, "packed_offset", torch.int32, E + 1, dev)
    return shape[:-1], dev


def _expert_call(fn: str, E, H, n, lead, packed_offset, pairs, head, count, tail, stream):
    """One call of an experts' bf16 product: `head` are the arguments in front of expert_count."""
    if packed_offset is None:
        _call(fn, _shape(pairs, H, E, 1, lead[1], 1), n, *head, count, *tail, stream=stream)
    else:
        _call(fn + "_packed", _shape(pairs, H, E, 1, 1, 1), lead[0], n, *head, count, packed_offset,
              *tail, stream=stream)


def _expert_gemm(x, count, offset, w, pairs, y, stream):
    E, N, H = _weights3(w, "w")
    lead, dev = _expert_rows(x, "recv", E, count, offset)
    _rows(x, "recv", (*lead, H), dev)
    _rows(w, "w", w.shape, dev)
    y = _new((*lead, N), _bf16(x), dev, stream) if y is None else y
    _rows(y, "y", (*lead, N), dev)
    _expert_call("ep_expert_gemm", E, H, N, lead, offset, pairs, (x,), count, (w, y), stream)
    return y


def ep_expert_gemm(recv: torch.Tensor, expert_count: torch.Tensor, w: torch.Tensor, pairs: int, *,
                   y=None, stream=None):
    """The experts' product on a padded bf16 receive buffer ``recv`` [E, C, H] (as ep_dispatch
    writes it), the first ``expert_count[e]`` rows of each expert: weights ``w`` [E, N, H] ->
    ``y`` [E, C, N] bf16. Rows that hold no pair are neither read nor written. ``pairs``: T * K, the
    pairs the layout placed (chooses the kernel and its grid, so that the order of the fp32 sums may
    differ, but not the rows that are computed; 0: no rows)."""
    return _expert_gemm(recv, expert_count, None, w, pairs, y, stream)


def ep_expert_gemm_packed(recv: torch.Tensor, expert_count: torch.Tensor,
                          packed_offset: torch.Tensor, w: torch.Tensor, pairs: int, *, y=None,
                          stream=None):
    """ep_expert_gemm on a packed buffer: ``recv`` [rows, H], expert e's rows from
    ``packed_offset[e]`` on -> ``y`` [rows, N] bf16."""
    return _expert_gemm(recv, expert_count, packed_offset, w, pairs, y, stream)


def _expert_swiglu(x, count, offset, w13, pairs, h, gu, stream):
    E, n, H = _weights3(w13, "w13")
    if n % 2:
        raise ValueError(f"w13: expected an even number of rows (gate, then up), got {n}")
    lead, dev = _expert_rows(x, "recv", E, count, offset)
    _rows(x, "recv", (*lead, H), dev)
    _rows(w13, "w13", w13.shape, dev)
    h = _new((*lead, n // 2), _bf16(x), dev, stream) if h is None else h
    _rows(h, "h", (*lead, n // 2), dev)
    if gu is not None:
        _rows(gu, "gu", (*lead, n), dev)
    _expert_call("ep_expert_swiglu", E, H, n // 2, lead, offset, pairs, (x,), count, (w13, gu, h),
                 stream)
    return h


def ep_expert_swiglu(recv: torch.Tensor, expert_count: torch.Tensor, w13: torch.Tensor, pairs: int,
                     *, h=None, gu=None, stream=None):
    """The gate and up products and SwiGLU on a padded bf16 receive buffer: ``recv`` [E, C, H],
    ``w13`` [E, 2I, H] (the I gate rows, then the I up rows) -> ``h`` [E, C, I] bf16, which
    ep_expert_gemm takes as its rows. ``gu`` [E, C, 2I] bf16, if given, receives the two products,
    which ep_expert_swiglu_dgrad needs."""
    return _expert_swiglu(recv, expert_count, None, w13, pairs, h, gu, stream)


def ep_expert_swiglu_packed(recv: torch.Tensor, expert_count: torch.Tensor,
                            packed_offset: torch.Tensor, w13: torch.Tensor, pairs: int, *, h=None,
                            gu=None, stream=None):
    """ep_expert_swiglu on a packed buffer: ``recv`` [rows, H] -> ``h`` [rows, I], ``gu``
    [rows, 2I]."""
    return _expert_swiglu(recv, expert_count, packed_offset, w13, pairs, h, gu, stream)


def _expert_dgrad(dy, count, offset, w, pairs, dx, stream):
    E, N, H = _weights3(w, "w")
    lead, dev = _expert_rows(dy, "dy", E, count, offset)
    _rows(dy, "dy", (*lead, N), dev)
    _rows(w, "w", w.shape, dev)
    dx = _new((*lead, H), _bf16(dy), dev, stream) if dx is None else dx
    _rows(dx, "dx", (*lead, H), dev)
    _expert_call("ep_expert_gemm_dgrad", E, H, N, lead, offset, pairs, (dy,), count, (w, dx), stream)
    return dx


def ep_expert_gemm_dgrad(dy: torch.Tensor, expert_count: torch.Tensor, w: torch.Tensor, pairs: int,
                         *, dx=None, stream=None):
    """The gradient of ep_expert_gemm's rows: ``dy`` [E, C, N], the forward call's ``w`` [E, N, H] ->
    ``dx`` [E, C, H] bf16. ep_combine of ``dx`` with weights 1 is the gradient of the token rows."""
    return _expert_dgrad(dy, expert_count, None, w, pairs, dx, stream)


def ep_expert_gemm_dgrad_packed(dy: torch.Tensor, expert_count: torch.Tensor,
                                packed_offset: torch.Tensor, w: torch.Tensor, pairs: int, *,
                                dx=None, stream=None):
    """ep_expert_gemm_dgrad on a packed buffer: ``dy`` [rows, N] -> ``dx`` [rows, H]."""
    return _expert_dgrad(dy, expert_count, packed_offset, w, pairs, dx, stream)


def _expert_swiglu_dgrad(dy, count, offset, w2, gu, pairs, dgu, stream):
    E, H, I = _weights3(w2, "w2")
    lead, dev = _expert_rows(dy, "dy", E, count, offset)
    _rows(dy, "dy", (*lead, H), dev)
    _rows(w2, "w2", w2.shape, dev)
    _rows(gu, "gu", (*lead, 2 * I), dev)
    dgu = _new((*lead, 2 * I), _bf16(dy), dev, stream) if dgu is None else dgu
    _rows(dgu, "dgu", (*lead, 2 * I), dev)
    _expert_call("ep_expert_swiglu_dgrad", E, H, I, lead, offset, pairs, (dy,), count, (w2, gu, dgu),
                 stream)
    return dgu


def ep_expert_swiglu_dgrad(dy: torch.Tensor, expert_count: torch.Tensor, w2: torch.Tensor,
                           gu: torch.Tensor, pairs: int, *, dgu=None, stream=None):
    """Back through the down projection and SwiGLU: ``dy`` [E, C, H], the gradient of the
    projection's output, its weights ``w2`` [E, H, I] and ``gu`` [E, C, 2I] as ep_expert_swiglu kept
    it -> ``dgu`` [E, C, 2I] bf16 (may be ``gu`` itself), whose ep_expert_gemm_dgrad and
    ep_expert_gemm_wgrad are the gradients of the gate and up products."""
    return _expert_swiglu_dgrad(dy, expert_count, None, w2, gu, pairs, dgu, stream)


def ep_expert_swiglu_dgrad_packed(dy: torch.Tensor, expert_count: torch.Tensor,
                                  packed_offset: torch.Tensor, w2: torch.Tensor, gu: torch.Tensor,
                                  pairs: int, *, dgu=None, stream=None):
    """ep_expert_swiglu_dgrad on a packed buffer: ``dy`` [rows, H], ``gu`` and ``dgu`` [rows, 2I]."""
    return _expert_swiglu_dgrad(dy, expert_count, packed_offset, w2, gu, pairs, dgu, stream)


def _expert_wgrad(dy, x, count, offset, pairs, dw, accumulate, stream):
    E = _experts(count)
    lead, dev = _expert_rows(dy, "dy", E, count, offset)
    N, H = dy.shape[-1], x.shape[-1]
    _rows(dy, "dy", (*lead, N), dev)
    _rows(x, "recv", (*lead, H), dev)
    if dw is None:
        if accumulate:
            raise ValueError("dw: accumulate adds to a float32 dw that the caller passes in")
        dw = _new((E, N, H), _bf16(dy), dev, stream)
    if tuple(dw.shape) != (E, N, H):
        raise ValueError(f"dw: expected {(E, N, H)}, got {tuple(dw.shape)}")
    f32 = dw.dtype == torch.float32
    if accumulate and not f32:
        raise TypeError(f"dw: accumulate needs torch.float32, got {dw.dtype}")
    _need(dw, "dw", torch.float32 if f32 else _bf16(dw), E * N * H, dev)
    fn = "ep_expert_gemm_wgrad_f32" if f32 else "ep_expert_gemm_wgrad"
    head = (int(bool(accumulate)), dy, x) if f32 else (dy, x)
    _expert_call(fn, E, H, N, lead, offset, pairs, head, count, (dw,), stream)
    return dw


def ep_expert_gemm_wgrad(dy: torch.Tensor, recv: torch.Tensor, expert_count: torch.Tensor,
                         pairs: int, *, dw=None, accumulate=False, stream=None):
    """The gradient of an experts' product's weights: ``dy`` [E, C, N] and the product's rows ``recv``
    [E, C, H] -> ``dw`` [E, N, H], all of it (zeros for an expert without rows). bf16, or float32 if
    such a ``dw`` is passed in; then ``accumulate`` adds to what it holds."""
    return _expert_wgrad(dy, recv, expert_count, None, pairs, dw, accumulate, stream)


def ep_expert_gemm_wgrad_packed(dy: torch.Tensor, recv: torch.Tensor, expert_count: torch.Tensor,
                                packed_offset: torch.Tensor, pairs: int, *, dw=None,
                                accumulate=False, stream=None):
    """ep_expert_gemm_wgrad on packed buffers: ``dy`` [rows, N], ``recv`` [rows, H]."""
    return _expert_wgrad(dy, recv, expert_count, packed_offset, pairs, dw, accumulate, stream)


def _combine_grad(dout, y, idx, slot, topk_w, dy, dtopk_w, stream):
    dev = dout.device
    (T, H), K = dout.shape, idx.shape[1]
    lead = tuple(y.shape[:-1])
    dy = _new(y.shape, _bf16(y), dev, stream) if dy is None else dy
    dtopk_w = _new((T, K), torch.float32, dev, stream) if dtopk_w is None else dtopk_w
    _rows(dout, "dout", (T, H), dev)
    _rows(y, "y", (*lead, H), dev)
    _rows(dy, "dy", (*lead, H), dev)
    for name, t, dtype in (("topk_idx", idx, torch.int32), ("slot", slot, torch.int32),
                           ("topk_w", topk_w, torch.float32), ("dtopk_w", dtopk_w, torch.float32)):
        _need(t, name, dtype, T * K, dev)
    return T, H, K, dy, dtopk_w


def ep_combine_grad(dout: torch.Tensor, y: torch.Tensor, topk_idx: torch.Tensor, slot: torch.Tensor,
                    topk_w: torch.Tensor, C: int, *, dy=None, dtopk_w=None, stream=None):
    """The gradient of ep_combine: ``dout`` [T, H] bf16 and the forward call's ``y`` [E, C, H],
    ``topk_idx``, ``slot`` and ``topk_w`` [T, K] -> ``dy`` [E, C, H] bf16, the rows that hold a pair
    (others keep what they hold), and ``dtopk_w`` [T, K] float32 (0 for a pair that is not kept)."""
    if dout.dim() != 2 or topk_idx.dim() != 2 or y.dim() != 3 or y.shape[1] != C:
        raise ValueError(f"expected dout [T, H], topk_idx [T, K] and y [E, {C}, H], got "
                         f"{tuple(dout.shape)}, {tuple(topk_idx.shape)} and {tuple(y.shape)}")
    T, H, K, dy, dtopk_w = _combine_grad(dout, y, topk_idx, slot, topk_w, dy, dtopk_w, stream)
    _call("ep_combine_grad", _shape(T, H, y.shape[0], K, C, 1), dout, y, topk_idx, slot, topk_w, dy,
          dtopk_w, stream=stream)
    return dy, dtopk_w


def ep_combine_grad_packed(dout: torch.Tensor, y: torch.Tensor, topk_idx: torch.Tensor,
                           slot: torch.Tensor, packed_offset: torch.Tensor, topk_w: torch.Tensor,
                           E: int, C: int, *, dy=None, dtopk_w=None, stream=None):
    """ep_combine_grad on packed buffers: ``y`` and ``dy`` [rows, H]."""
    if dout.dim() != 2 or topk_idx.dim() != 2 or y.dim() != 2:
        raise ValueError(f"expected dout [T, H], topk_idx [T, K] and y [rows, H], got "
                         f"{tuple(dout.shape)}, {tuple(topk_idx.shape)} and {tuple(y.shape)}")
    T, H, K, dy, dtopk_w = _combine_grad(dout, y, topk_idx, slot, topk_w, dy, dtopk_w, stream)
    _need(packed_offset, "packed_offset", torch.int32, E + 1, dout.device)
    _call("ep_combine_grad_packed", _shape(T, H, E, K, C, 1), y.shape[0], dout, y, topk_idx, slot,
          packed_offset, topk_w, dy, dtopk_w, stream=stream)
    return dy, dtopk_w


# ------------------------------------------------------------------------------------------
# the dense product beside the experts
# ------------------------------------------------------------------------------------------

def _activation(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act: expected one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _linear_args(x, w, act):
    xs, ws, dev = x.shape, w.shape, x.device
    if len(xs) != 2 or len(ws) != 2 or xs[1] != ws[1]:
        raise ValueError(f"expected x [T, H] and w [N, H], got {tuple(xs)} and {tuple(ws)}")
    a = _activation(act)
    _rows(x, "x", xs, dev)
    _rows(w, "w", ws, dev)
    return xs[0], xs[1], ws[0], a, dev


def ep_linear(x: torch.Tensor, w: torch.Tensor, *, bias=None, act="none", residual=None, pre=None,
              out=None, stream=None):
    """``out = act(x @ w.T + bias) + residual``, one rounding: ``x`` [T, H], ``w`` [N, H], ``bias`` [N]
    and ``residual`` [T, N] (or None) bf16 -> ``out`` [T, N] bf16 (may be ``residual`` itself). ``act``:
    "none", "relu", "silu" or "gelu" (with the normal distribution). ``pre`` [T, N] bf16, if given,
    receives ``x @ w.T + bias``, which ep_linear_grad needs for an activation."""
    T, H, N, a, dev = _linear_args(x, w, act)
    out = _new((T, N), _bf16(x), dev, stream) if out is None else out
    if bias is not None:
        _rows(bias, "bias", (N,), dev)
    _rows(out, "out", (T, N), dev)
    if residual is not None:
        _rows(residual, "residual", (T, N), dev)
    if pre is not None:
        _rows(pre, "pre", (T, N), dev)
    _call("ep_linear", _shape(T, H, 1, 1, 1, 1), N, a, x, w, bias, residual, pre, out, stream=stream)
    return out


def linear_grad_workspace_bytes(T: int, N: int, act: str) -> int:
    """Bytes of workspace ep_linear_grad needs for T rows, N outputs and an activation."""
    _fits32("ep_linear_grad_workspace_bytes", N)
    return int(load_library().ep_linear_grad_workspace_bytes(
        ctypes.byref(_shape(T, 8, 1, 1, 1, 1)), N, _activation(act)))


def ep_linear_grad(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *, act="none", pre=None,
                   dx=None, dw=None, dbias=None, workspace=None, stream=None):
    """The gradients of ep_linear: ``dout`` [T, N] bf16 and the forward call's ``x``, ``w``, ``act`` and
    (with an activation) ``pre`` -> ``dx`` [T, H] bf16, ``dw`` [N, H] bf16, ``dbias`` [N] float32. The
    residual's gradient is ``dout``. ``workspace``: a device tensor of at least
    linear_grad_workspace_bytes(T, N, act) bytes (allocated here if not given)."""
    T, H, N, a, dev = _linear_args(x, w, act)
    _rows(dout, "dout", (T, N), dev)
    if (pre is None) != (act == "none"):
        raise ValueError("pre: given exactly for an activation")
    if pre is not None:
        _rows(pre, "pre", (T, N), dev)
    dx = _new((T, H), _bf16(x), dev, stream) if dx is None else dx
    dw = _new((N, H), _bf16(x), dev, stream) if dw is None else dw
    dbias = _new((N,), torch.float32, dev, stream) if dbias is None else dbias
    _rows(dx, "dx", (T, H), dev)
    _rows(dw, "dw", (N, H), dev)
    _need(dbias, "dbias", torch.float32, N, dev)
    if workspace is None:
        workspace = _own_workspace(linear_grad_workspace_bytes(T, N, act), dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous tensor on the rows' device")
    _call("ep_linear_grad", _shape(T, H, 1, 1, 1, 1), N, a, dout, pre, x, w, dx, dw, dbias, workspace,
          workspace.numel() * workspace.element_size(), stream=stream)
    return dx, dw, dbias


def ep_check_e4m3_conversion(first_pattern: int, count: int, *, device=None, stream=None):
    """Compare the FP8 cast's two E4M3 encoders (the hardware conversion and the software
    one) on the fp32 bit patterns [first_pattern, first_pattern + count) on the current
    device. Returns (mismatches, smallest mismatching pattern or None) after synchronising."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    res = _new(2, torch.int32, dev, stream)
    _require_current("ep_check_e4m3_conversion", dev)
    L = load_library()
    rc = L.ep_check_e4m3_conversion(first_pattern, count, res.data_ptr(), res.data_ptr() + 4,
                                    _stream(stream))
    _check("ep_check_e4m3_conversion", rc)
    torch.cuda.synchronize(dev)
    n, first = (int(v) & 0xFFFFFFFF for v in res.cpu().tolist())
    return n, (None if n == 0 else first)


_resources = None


def kernel_resources() -> dict:
    """The compiler's resource figures per kernel symbol, written by the build beside the
    library (empty if that file is missing)."""
    global _resources
    if _resources is None:
        import json
        path = os.path.join(os.path.dirname(library_path()), "kernel_resources.json")
        try:
            with open(path) as f:
                _resources = json.load(f).get("kernels", {})
        except (OSError, ValueError):
            _resources = {}
    return _resources


def last_launches() -> list:
    """The kernel launches of this thread's most recent library call: per launch the kernel
    symbol, grid and workgroup sizes, LDS, and the register figures of the runtime and of the
    compiler's report."""
    L = load_library()
    recs = (EpLaunchRecord * 8)()
    n = L.ep_last_launches(recs, 8)
    res = kernel_resources()
    out = []
    for r in recs[:min(n, 8)]:
        name = (r.kernel or b"").decode()
        d = {"kernel": name, "grid": [r.grid_x, r.grid_y, r.grid_z],
             "block": [r.block_x, r.block_y, r.block_z],
             "dynamic_lds_bytes": r.dynamic_lds_bytes, "static_lds_bytes": r.static_lds_bytes,
             "vgprs": r.vgprs, "private_bytes": r.private_bytes}
        if name in res:
            d["compiler"] = res[name]
        out.append(d)
    return out
