"""Python binding of liba2av.so (include/a2av.h), argument marshalling only.

Every function has the name of the C entry point it calls and takes torch tensors (or
raw device addresses as ints) where the C call takes device pointers; the stream
defaults to torch's current stream.  No step of the path runs in Python: the library is
required, and a missing build raises at import of the first call.
"""
import ctypes
import functools
import os

import torch

F32 = 0
BF16 = 1
MX8 = 2
MX4 = 3
OK = 0
ERR_INVALID = -1
ERR_NOMEM = -2
ERR_HIP = -3
ERR_SCRATCH = -4
NOALLOC_MAX_RANKS = 256
NOALLOC_SCRATCH_BYTES = 1 << 20
ST_EXPERT_RANGE = 1
ST_RECV_OVERFLOW = 2
ST_BOUNDS = 4
ST_OFFSETS = 8
ACT_NONE = 0
ACT_SWIGLU = 1
EXPERT_IDENTITY = 0
EXPERT_SCALE = 1
PATH_STAGED = 0
PATH_DIRECT = 1
LAYOUT_SOURCE_MAJOR = 0
LAYOUT_EXPERT_MAJOR = 1
STAGES = 5
STREAM_READ = 0
STREAM_WRITE = 1
STREAM_READ_OUT_BYTES = 1 << 20
STAGE_NAMES = ("plan", "pack", "exchange", "return", "combine")

# A2AV_DEBUG=1 in the environment selects the debug build (device-side bounds checks,
# status bit ST_BOUNDS); same exports and results.
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "liba2av_debug.so" if os.environ.get("A2AV_DEBUG") == "1" else "liba2av.so")
EXPORTS = ("a2av_create", "a2av_destroy", "a2av_workspace_bytes", "a2av_dispatch", "a2av_combine",
           "a2av_alltoallv", "a2av_alltoallv_noalloc", "a2av_copy_positions", "a2av_copy_recv_expert_offsets",
           "a2av_copy_send_offsets", "a2av_recv_expert_offsets", "a2av_row_bytes", "a2av_rmsnorm",
           "a2av_expert_matmul", "a2av_expert_apply", "a2av_route_step", "a2av_copy_reference",
           "a2av_stream_reference", "a2av_timing_begin", "a2av_timing_end", "a2av_error_string")

# 8-bit rows and 4- and 8-bit weights are bytes
TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16, MX8: torch.uint8, MX4: torch.uint8}


class Config(ctypes.Structure):
    _fields_ = [("num_ranks", ctypes.c_int32), ("tokens_per_rank", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("experts_per_rank", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("recv_capacity_rows", ctypes.c_int64), ("path", ctypes.c_int32), ("recv_layout", ctypes.c_int32)]


class Matmul(ctypes.Structure):
    _fields_ = [("num_ranks", ctypes.c_int32), ("experts_per_rank", ctypes.c_int32),
                ("capacity_rows", ctypes.c_int64), ("k", ctypes.c_int32), ("n", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class A2AVError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {code} ({error_string(code)})")
        self.code = code


_lib = None


def lib():
    """The loaded library.  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with moe_alltoallv_resident_amd/build.py "
                               "(or __graft_entry__.build()); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.a2av_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(vp)]
        L.a2av_destroy.argtypes = [vp]
        L.a2av_workspace_bytes.argtypes = [ctypes.POINTER(Config)]
        L.a2av_workspace_bytes.restype = i64
        L.a2av_dispatch.argtypes = [vp] * 9
        L.a2av_combine.argtypes = [vp] * 6
        L.a2av_alltoallv.argtypes = [vp] * 8
        L.a2av_alltoallv_noalloc.argtypes = [ctypes.POINTER(Config)] + [vp] * 7
        L.a2av_copy_positions.argtypes = [vp, vp, vp]
        L.a2av_copy_send_offsets.argtypes = [vp, vp, vp]
        L.a2av_copy_recv_expert_offsets.argtypes = [vp, vp, vp]
        L.a2av_recv_expert_offsets.argtypes = [vp]
        L.a2av_recv_expert_offsets.restype = vp
        L.a2av_row_bytes.argtypes = [i32, i64]
        L.a2av_row_bytes.restype = i64
        L.a2av_rmsnorm.argtypes = [vp] * 6 + [i64, i32, i32, ctypes.c_float, vp]
        L.a2av_expert_matmul.argtypes = [ctypes.POINTER(Matmul)] + [vp] * 7
        L.a2av_expert_apply.argtypes = [vp, vp, vp, i32, vp]
        L.a2av_route_step.argtypes = [vp, vp, i32, i64, vp, vp, vp, vp]
        L.a2av_copy_reference.argtypes = [vp, vp, i64, i64, vp]
        L.a2av_stream_reference.argtypes = [vp, vp, i64, i32, vp]
        L.a2av_timing_begin.argtypes = [vp, i32]
        L.a2av_timing_end.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i32)]
        L.a2av_error_string.argtypes = [ctypes.c_int]
        L.a2av_error_string.restype = ctypes.c_char_p
        for f in EXPORTS:
            if f not in ("a2av_workspace_bytes", "a2av_error_string", "a2av_recv_expert_offsets", "a2av_row_bytes"):
                getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def error_string(code: int) -> str:
    return lib().a2av_error_string(code).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("device tensors must be contiguous GPU tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(stream)


def _check(fn, rc):
    if rc != OK:
        raise A2AVError(fn, rc)


def make_config(num_ranks, tokens_per_rank, hidden, dtype, experts_per_rank, top_k, recv_capacity_rows=0,
                path=PATH_STAGED, recv_layout=LAYOUT_SOURCE_MAJOR) -> Config:
    return Config(num_ranks, tokens_per_rank, hidden, dtype, experts_per_rank, top_k, recv_capacity_rows, path,
                  recv_layout)


def a2av_workspace_bytes(cfg: Config) -> int:
    return lib().a2av_workspace_bytes(ctypes.byref(cfg))


def a2av_create(cfg: Config) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check("a2av_create", lib().a2av_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h


def a2av_destroy(h) -> None:
    _check("a2av_destroy", lib().a2av_destroy(h))


def a2av_dispatch(h, x, topk_ids, recv, split, recv_counts, recv_offsets, status, stream=None) -> None:
    _check("a2av_dispatch", lib().a2av_dispatch(h, _ptr(x), _ptr(topk_ids), _ptr(recv), _ptr(split),
                                                _ptr(recv_counts), _ptr(recv_offsets), _ptr(status),
                                                _stream(stream)))


def a2av_combine(h, expert_out, gates, y, status, stream=None) -> None:
    _check("a2av_combine", lib().a2av_combine(h, _ptr(expert_out), _ptr(gates), _ptr(y), _ptr(status),
                                              _stream(stream)))


def a2av_alltoallv(h, send, send_counts, recv, recv_counts, recv_offsets, status, stream=None) -> None:
    _check("a2av_alltoallv", lib().a2av_alltoallv(h, _ptr(send), _ptr(send_counts), _ptr(recv),
                                                  _ptr(recv_counts), _ptr(recv_offsets), _ptr(status),
                                                  _stream(stream)))


def a2av_alltoallv_noalloc(cfg: Config, send, send_counts, recv, recv_counts, recv_offsets, status,
                           stream=None) -> None:
    _check("a2av_alltoallv_noalloc",
           lib().a2av_alltoallv_noalloc(ctypes.byref(cfg), _ptr(send), _ptr(send_counts), _ptr(recv),
                                        _ptr(recv_counts), _ptr(recv_offsets), _ptr(status), _stream(stream)))


def a2av_copy_positions(h, pos, stream=None) -> None:
    _check("a2av_copy_positions", lib().a2av_copy_positions(h, _ptr(pos), _stream(stream)))


def a2av_copy_recv_expert_offsets(h, recv_expert_offsets, stream=None) -> None:
    _check("a2av_copy_recv_expert_offsets",
           lib().a2av_copy_recv_expert_offsets(h, _ptr(recv_expert_offsets), _stream(stream)))


def a2av_copy_send_offsets(h, send_offsets, stream=None) -> None:
    _check("a2av_copy_send_offsets", lib().a2av_copy_send_offsets(h, _ptr(send_offsets), _stream(stream)))


def a2av_recv_expert_offsets(h) -> int:
    """Device address of the handle's own table of group starts (expert-major handles)."""
    return lib().a2av_recv_expert_offsets(h)


def a2av_row_bytes(dtype: int, n: int) -> int:
    return lib().a2av_row_bytes(dtype, n)


def a2av_rmsnorm(x, residual, weight, residual_out, y, y8, rows, hidden, dtype, eps, stream=None) -> None:
    _check("a2av_rmsnorm", lib().a2av_rmsnorm(_ptr(x), _ptr(residual), _ptr(weight), _ptr(residual_out), _ptr(y),
                                              _ptr(y8), rows, hidden, dtype, eps, _stream(stream)))


def a2av_expert_matmul(cfg: Matmul, inp, expert_offsets, weight, weight_scales, out, status, stream=None) -> None:
    _check("a2av_expert_matmul",
           lib().a2av_expert_matmul(ctypes.byref(cfg), _ptr(inp), _ptr(expert_offsets), _ptr(weight),
                                    _ptr(weight_scales), _ptr(out), _ptr(status), _stream(stream)))


def a2av_expert_apply(h, inp, out, mode, stream=None) -> None:
    _check("a2av_expert_apply", lib().a2av_expert_apply(h, _ptr(inp), _ptr(out), mode, _stream(stream)))


def a2av_route_step(ids_table, gates_table, steps, n, counter, ids, gates, stream=None) -> None:
    _check("a2av_route_step", lib().a2av_route_step(_ptr(ids_table), _ptr(gates_table), steps, n, _ptr(counter),
                                                    _ptr(ids), _ptr(gates), _stream(stream)))


def a2av_copy_reference(src, dst, rows, row_bytes, stream=None) -> None:
    _check("a2av_copy_reference", lib().a2av_copy_reference(_ptr(src), _ptr(dst), rows, row_bytes, _stream(stream)))


def _nbytes(t):
    return t.numel() * t.element_size() if isinstance(t, torch.Tensor) else None


def a2av_stream_reference(src, dst, nbytes, mode, stream=None) -> None:
    # the kernels write a fixed-size result (read) or nbytes (write): short tensors are
    # refused here rather than written past their end
    need_dst = STREAM_READ_OUT_BYTES if mode == STREAM_READ else nbytes
    if _nbytes(dst) is not None and _nbytes(dst) < need_dst:
        raise ValueError(f"a2av_stream_reference: dst holds {_nbytes(dst)} bytes, needs {need_dst}")
    if mode == STREAM_READ and _nbytes(src) is not None and _nbytes(src) < nbytes:
        raise ValueError(f"a2av_stream_reference: src holds {_nbytes(src)} bytes, reads {nbytes}")
    _check("a2av_stream_reference", lib().a2av_stream_reference(_ptr(src), _ptr(dst), nbytes, mode, _stream(stream)))


def a2av_timing_begin(h, max_calls) -> None:
    _check("a2av_timing_begin", lib().a2av_timing_begin(h, max_calls))


def a2av_timing_end(h):
    """Returns (ms_sum[5], launches[5]) per stage: plan, pack, exchange, return, combine."""
    ms = (ctypes.c_double * STAGES)()
    n = (ctypes.c_int32 * STAGES)()
    _check("a2av_timing_end", lib().a2av_timing_end(h, ms, n))
    return list(ms), list(n)


# The checks below are host-side only (no synchronisation), as Session's, and written for small
# calls, where they take longer than the kernels.

def _check_device(name, t, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}: every tensor must be on one GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_like(name, t, dev, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        _check_device(name, t, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _address(t):
    return None if t is None else t.data_ptr()


# the current stream's address without the Stream object around it, where torch offers that
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(name, dev, stream, call):
    """call(stream) with `dev` the current GPU, on the given stream or that GPU's current one."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch(name, dev, stream, call)
    if stream is None:
        stream = _current_stream(dev)
    rc = call(stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream)
    if rc != OK:
        raise A2AVError(name, rc)


_ROWS_DTYPE = {torch.float32: F32, torch.bfloat16: BF16}


def rmsnorm(x, weight, eps, residual=None, residual_out=None, y=None, y8=None, stream=None) -> None:
    """a2av_rmsnorm on torch tensors, with their types and sizes checked.

    x [..., hidden] float32 or bfloat16 (weight, residual, residual_out, y alike); y8 uint8
    [..., a2av_row_bytes(MX8, hidden)].  weight may be None (ones).  The outputs given are
    written; at least one is.
    """
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    dtype, shape, dev = x.dtype, x.shape, x.get_device()
    code = _ROWS_DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"x has dtype {dtype}, expected float32 or bfloat16")
    if not shape:
        raise ValueError("x must have at least one dimension")
    hidden = shape[-1]
    _check_device("x", x, dev)
    if weight is not None:
        _check_like("weight", weight, dev, dtype, (hidden,))
    if residual is not None:
        _check_like("residual", residual, dev, dtype, shape)
    if residual_out is not None:
        _check_like("residual_out", residual_out, dev, dtype, shape)
    if y is not None:
        _check_like("y", y, dev, dtype, shape)
    if y8 is not None:
        _check_like("y8", y8, dev, torch.uint8, shape[:-1] + (a2av_row_bytes(MX8, hidden),))
    rows = x.numel() // hidden if hidden else 0
    _launch("a2av_rmsnorm", dev, stream, lambda st: lib().a2av_rmsnorm(
        x.data_ptr(), _address(residual), _address(weight), _address(residual_out), _address(y), _address(y8), rows, hidden,
        code, eps, st))


@functools.lru_cache(maxsize=1024)
def _matmul_plan(R, epr, cap, k, n, in_dtype, weight_dtype, out_dtype, activation):
    """The call's description and the row lengths (in elements of the tensors) that it asks for."""
    for name, d in (("in_dtype", in_dtype), ("weight_dtype", weight_dtype), ("out_dtype", out_dtype)):
        if d not in TORCH_DTYPE or (d == MX4 and name != "weight_dtype"):
            raise ValueError(f"{name} {d} is not an element type of this argument")
    width = n // 2 if activation == ACT_SWIGLU else n
    return (ctypes.byref(Matmul(R, epr, cap, k, n, in_dtype, weight_dtype, out_dtype, activation)),
            (R, cap, a2av_row_bytes(MX8, k) if in_dtype == MX8 else k),
            (R, cap, a2av_row_bytes(MX8, width) if out_dtype == MX8 else width))


def _expert_matmul(dev, R, epr, cap, inp, offsets, weight, out, status, weight_scales, in_dtype, weight_dtype, out_dtype,
                   activation, stream):
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch tensor")
    if weight.dim() != 3:
        raise ValueError(f"weight has {weight.dim()} dimensions, expected 3")
    _, n, w_row = weight.shape
    k = w_row * 2 if weight_dtype == MX4 else w_row
    cfg, in_shape, out_shape = _matmul_plan(R, epr, cap, k, n, in_dtype, weight_dtype, out_dtype, activation)
    _check_like("weight", weight, dev, TORCH_DTYPE[weight_dtype], (R * epr, n, w_row))
    _check_like("inp", inp, dev, TORCH_DTYPE[in_dtype], in_shape)
    _check_like("out", out, dev, TORCH_DTYPE[out_dtype], out_shape)
    if weight_scales is not None:
        _check_like("weight_scales", weight_scales, dev, torch.uint8, (R * epr, n, k // 32))
    _check_device("status", status, dev)
    if status.dtype != torch.int32 or status.numel() < 1:
        raise TypeError("status must be an int32 tensor of one element")
    _launch("a2av_expert_matmul", dev, stream, lambda st: lib().a2av_expert_matmul(
        cfg, inp.data_ptr(), offsets, weight.data_ptr(), _address(weight_scales), out.data_ptr(), status.data_ptr(), st))


def expert_matmul(inp, expert_offsets, weight, out, status, weight_scales=None, in_dtype=BF16, weight_dtype=BF16,
                  out_dtype=BF16, activation=ACT_NONE, stream=None) -> None:
    """a2av_expert_matmul on torch tensors, with their types and sizes checked.

    inp [R][cap][row] and out [R][cap][row] (MX8: uint8 rows of a2av_row_bytes);
    expert_offsets int32 [R][epr + 1]; weight [R * epr][n][k] (MX4: uint8 [..][k / 2]; MX8:
    uint8); weight_scales uint8 [R * epr][n][k / 32] for MX4 and MX8; status int32 [1].
    """
    if not isinstance(inp, torch.Tensor) or not isinstance(expert_offsets, torch.Tensor):
        raise TypeError("inp and expert_offsets must be torch tensors")
    if expert_offsets.dim() != 2 or inp.dim() != 3:
        raise ValueError("expert_offsets must be [R][epr + 1] and inp [R][cap][row]")
    R, starts = expert_offsets.shape
    dev = inp.get_device()
    _check_like("expert_offsets", expert_offsets, dev, torch.int32, (inp.shape[0], starts))
    _expert_matmul(dev, R, starts - 1, inp.shape[1], inp, expert_offsets.data_ptr(), weight, out, status, weight_scales,
                   in_dtype, weight_dtype, out_dtype, activation, stream)


class Session:
    """A handle plus the caller-owned device buffers of one configuration.

    dtype MX8: x and recv are 8-bit rows [..][a2av_row_bytes(MX8, H)] (uint8), the experts'
    outputs and y bfloat16.  Allocates (once) recv [R][cap][H], split [R][E], recv_counts [R][R],
    recv_offsets [R][R+1] and status on the current GPU; dispatch/combine then only
    enqueue library calls, so they can be captured in a graph.
    """

    def __init__(self, num_ranks, tokens_per_rank, hidden, dtype, experts_per_rank, top_k,
                 recv_capacity_rows=0, path=PATH_STAGED, recv_layout=LAYOUT_SOURCE_MAJOR, device="cuda"):
        self.cfg = make_config(num_ranks, tokens_per_rank, hidden, dtype, experts_per_rank, top_k,
                               recv_capacity_rows, path, recv_layout)
        self.path = path
        self.recv_layout = recv_layout
        self.epr = experts_per_rank
        self.R, self.T, self.H, self.k = num_ranks, tokens_per_rank, hidden, top_k
        self.E = num_ranks * experts_per_rank
        self.cap = recv_capacity_rows or num_ranks * tokens_per_rank * min(top_k, experts_per_rank)
        self.dtype = dtype
        self.torch_dtype = TORCH_DTYPE[dtype]
        # columns of a dispatched row, element type of a combined one
        self.cols = a2av_row_bytes(MX8, hidden) if dtype == MX8 else hidden
        self.out_dtype = torch.bfloat16 if dtype == MX8 else self.torch_dtype
        self.device = torch.device(device)
        with torch.cuda.device(self.device):
            self.handle = a2av_create(self.cfg)
        R = num_ranks
        self.recv = torch.empty((R, self.cap, self.cols), dtype=self.torch_dtype, device=self.device)
        self.split = torch.empty((R, self.E), dtype=torch.int32, device=self.device)
        self.recv_counts = torch.empty((R, R), dtype=torch.int32, device=self.device)
        self.recv_offsets = torch.empty((R, R + 1), dtype=torch.int32, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _check_tensor(self, name, t, dtype, numel):
        # host-side checks only (no synchronisation): a wrong element type or a short
        # buffer would otherwise be read or written past its end by the kernels
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.numel() != numel:
            raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
        if t.device != self.device and not (t.is_cuda and self.device.index is None):
            raise ValueError(f"{name} is on {t.device}, the session on {self.device}")

    def dispatch(self, x, topk_ids, stream=None):
        R, T, k = self.R, self.T, self.k
        self._check_tensor("x", x, self.torch_dtype, R * T * self.cols)
        self._check_tensor("topk_ids", topk_ids, torch.int32, R * T * k)
        a2av_dispatch(self.handle, x, topk_ids, self.recv, self.split, self.recv_counts, self.recv_offsets,
                      self.status, stream)
        return self.recv

    def expert(self, inp, out, mode, stream=None):
        n = self.R * self.cap * self.H
        self._check_tensor("expert input", inp, self.torch_dtype, n)
        self._check_tensor("expert output", out, self.torch_dtype, n)
        a2av_expert_apply(self.handle, inp, out, mode, stream)
        return out

    def combine(self, expert_out, gates, y, stream=None):
        R, T, H, k = self.R, self.T, self.H, self.k
        self._check_tensor("expert_out", expert_out, self.out_dtype, R * self.cap * H)
        self._check_tensor("gates", gates, torch.float32, R * T * k)
        self._check_tensor("y", y, self.out_dtype, R * T * H)
        a2av_combine(self.handle, expert_out, gates, y, self.status, stream)
        return y

    def expert_matmul(self, inp, weight, out, weight_scales=None, in_dtype=None, weight_dtype=BF16, out_dtype=BF16,
                      activation=ACT_NONE, stream=None):
        """The experts' products on rows of the latest dispatch (expert-major sessions): inp and out are
        [R][cap][row], the group starts are the handle's own table."""
        if self.recv_layout != LAYOUT_EXPERT_MAJOR:
            raise ValueError("expert_matmul needs an expert-major session")
        _expert_matmul(self.status.get_device(), self.R, self.epr, self.cap, inp, a2av_recv_expert_offsets(self.handle), weight,
                       out, self.status, weight_scales, self.dtype if in_dtype is None else in_dtype, weight_dtype, out_dtype,
                       activation, stream)
        return out

    def positions(self):
        pos = torch.empty((self.R, self.T, self.k), dtype=torch.int32, device=self.device)
        a2av_copy_positions(self.handle, pos)
        return pos

    def recv_expert_offsets(self):
        out = torch.empty((self.R, self.epr + 1), dtype=torch.int32, device=self.device)
        a2av_copy_recv_expert_offsets(self.handle, out)
        return out

    def send_offsets(self):
        so = torch.empty((self.R, self.R + 1), dtype=torch.int32, device=self.device)
        a2av_copy_send_offsets(self.handle, so)
        return so

    def close(self):
        if self.handle is not None:
            torch.cuda.synchronize(self.device)
            a2av_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
