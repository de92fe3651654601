"""Python binding of libmoonep.so: the balanced expert-parallel hot path on MI355X.

Argument marshalling only. Every step of the plan, dispatch, replicate, combine
and reduce runs in the HIP kernels of the library; torch provides device memory
and streams. The functions carry the C names and take the same arguments:
`dims` is a Dims, arrays are torch tensors on the GPU, `stream` is a
torch.cuda.Stream (default: the current stream of the tensors' device).

If the library has not been built this module raises ImportError: there is no
other implementation to fall back on.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
from typing import Dict, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoonep.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python -c 'import __graft_entry__ as g; g.build()' from the repository root)")

_lib = ctypes.CDLL(LIB_PATH)

F32 = 0
BF16 = 1
STATIC_SCRATCH_BYTES = 8 << 20  # MOONEP_STATIC_SCRATCH_BYTES
NORM_DOUBLES = 2049  # MOONEP_NORM_DOUBLES
OK, ERR_DIMS, ERR_PTR, ERR_HIP, ERR_SIZE = 0, -1, -2, -3, -4
STATUS_BAD_ID, STATUS_REPEAT_ID, STATUS_OVER_B = 1, 2, 4
OP_DISPATCH, OP_COMBINE = 1, 2
PLAN_BOUNDED, PLAN_FOUR_LAUNCH, PLAN_TWO_LAUNCH = 1, 2, 4

ENTRY_POINTS = ("moonep_plan_layout", "moonep_plan", "moonep_plan_ex", "moonep_plan_bounded",
                "moonep_plan_noscratch", "moonep_dispatch", "moonep_replicate",
                "moonep_combine", "moonep_reduce_dup_grads", "moonep_combine_backward",
                "moonep_dispatch_backward", "moonep_expert_matmul",
                "moonep_expert_matmul_wgrad", "moonep_quantize_rows",
                "moonep_expert_matmul_quant", "moonep_grad_sumsq", "moonep_grad_clip",
                "moonep_launch_count", "moonep_strerror")


class Dims(ctypes.Structure):
    """moonep_dims: R ranks, E experts, K per token, S tokens per rank, B duplicate
    slots per rank, dtype of hidden rows (F32/BF16), H hidden size."""
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32),
                ("S", ctypes.c_int32), ("B", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("H", ctypes.c_int64)]

    def __repr__(self):
        return (f"Dims(R={self.R}, E={self.E}, K={self.K}, S={self.S}, B={self.B}, "
                f"dtype={self.dtype}, H={self.H})")


_LAYOUT_OFFSETS = ("status", "maxT", "maxvio", "T", "hoff", "L", "keep", "O", "D", "Opre",
                   "Dpre", "dst", "src", "n_dup", "dup_expert", "dup_start", "dup_count",
                   "seg_ptr", "seg_expert", "n_list", "list_expert", "list_rank", "list_b",
                   "dup_ptr", "ws_tile_counts", "ws_tile_status", "ws_mat_pre", "ws_xlist",
                   "ws_n_x", "ws_piece_js", "ws_kept", "ws_koff", "ws_upre", "ws_pslot",
                   "ws_pcnt")


class Layout(ctypes.Structure):
    _fields_ = ([("bytes", ctypes.c_int64), ("persist_bytes", ctypes.c_int64),
                 ("dcap", ctypes.c_int32), ("pcap", ctypes.c_int32),
                 ("n_tiles", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
                 ("plan_launches", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in _LAYOUT_OFFSETS])


_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_P_DIMS, _P_LAY = ctypes.POINTER(Dims), ctypes.POINTER(Layout)
_lib.moonep_plan_layout.argtypes = [_P_DIMS, _P_LAY]
_lib.moonep_plan.argtypes = [_P_DIMS, _vp, _vp, _vp]
_lib.moonep_plan_bounded.argtypes = [_P_DIMS, _vp, _vp, _vp]
_lib.moonep_plan_ex.argtypes = [_P_DIMS, _vp, _vp, _i32, _vp]
_lib.moonep_plan_noscratch.argtypes = [_P_DIMS, _vp, _vp, _i32, _vp]
_lib.moonep_dispatch.argtypes = [_P_DIMS, _vp, _vp, _vp, _vp]
_lib.moonep_replicate.argtypes = [_P_DIMS, _vp, _vp, _vp, _i64, _vp]
_lib.moonep_combine.argtypes = [_P_DIMS, _vp, _vp, _vp, _vp, _i32, _vp]
_lib.moonep_reduce_dup_grads.argtypes = [_P_DIMS, _vp, _vp, _vp, _i64, _vp]
_lib.moonep_combine_backward.argtypes = [_P_DIMS, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.moonep_dispatch_backward.argtypes = [_P_DIMS, _vp, _vp, _vp, _i32, _vp]
_lib.moonep_expert_matmul.argtypes = [_P_DIMS, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]
_lib.moonep_expert_matmul_wgrad.argtypes = [_P_DIMS, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32,
                                            _vp]
_lib.moonep_quantize_rows.argtypes = [_i64, _i64, _vp, _i32, _vp, _vp, _vp]
_lib.moonep_expert_matmul_quant.argtypes = [_P_DIMS, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                            _i64, _i64, _i64, _vp]
_lib.moonep_grad_sumsq.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp]
_lib.moonep_grad_clip.argtypes = [_i32, _vp, _vp, _vp, _vp, _vp, ctypes.c_double, _vp, _vp]
_lib.moonep_launch_count.argtypes = [_P_DIMS, _i32, ctypes.POINTER(ctypes.c_int32)]
_lib.moonep_strerror.argtypes = [ctypes.c_int]
_lib.moonep_strerror.restype = ctypes.c_char_p
for _n in ENTRY_POINTS[:-1]:
    getattr(_lib, _n).restype = ctypes.c_int


class MoonEPError(RuntimeError):
    def __init__(self, rc: int, where: str):
        super().__init__(f"{where}: {moonep_strerror(rc)} (rc={rc})")
        self.rc = rc


def moonep_strerror(rc: int) -> str:
    return _lib.moonep_strerror(rc).decode()


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise MoonEPError(rc, where)


def _torch():
    import torch
    return torch


def _ptr(t, name: str, dtype=None, numel: Optional[int] = None) -> int:
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() * t.element_size() < numel:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs {numel}")
    return t.data_ptr()


def _stream(stream, ref) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(ref.device)
    return stream.cuda_stream


def _row_dtype(dims: Dims):
    torch = _torch()
    return torch.bfloat16 if dims.dtype == BF16 else torch.float32


def moonep_plan_layout(dims: Dims) -> Layout:
    lay = Layout()
    _check(_lib.moonep_plan_layout(ctypes.byref(dims), ctypes.byref(lay)), "moonep_plan_layout")
    return lay


def moonep_launch_count(dims: Dims, op: int) -> int:
    """Kernel launches one moonep_dispatch (OP_DISPATCH) or moonep_combine
    (OP_COMBINE, output in dims.dtype) call enqueues on the current device."""
    n = ctypes.c_int32(0)
    _check(_lib.moonep_launch_count(ctypes.byref(dims), op, ctypes.byref(n)), "moonep_launch_count")
    return int(n.value)


def moonep_plan(dims: Dims, topk_ids, plan_buf, stream=None) -> None:
    torch = _torch()
    lay = moonep_plan_layout(dims)
    ids = _ptr(topk_ids, "topk_ids", torch.int32, 4 * dims.R * dims.S * dims.K)
    pb = _ptr(plan_buf, "plan_buf", None, lay.bytes)
    _check(_lib.moonep_plan(ctypes.byref(dims), ids, pb, _stream(stream, plan_buf)), "moonep_plan")


def moonep_plan_bounded(dims: Dims, topk_ids, plan_buf, stream=None) -> None:
    torch = _torch()
    lay = moonep_plan_layout(dims)
    ids = _ptr(topk_ids, "topk_ids", torch.int32, 4 * dims.R * dims.S * dims.K)
    pb = _ptr(plan_buf, "plan_buf", None, lay.bytes)
    _check(_lib.moonep_plan_bounded(ctypes.byref(dims), ids, pb, _stream(stream, plan_buf)),
           "moonep_plan_bounded")


def moonep_plan_ex(dims: Dims, topk_ids, plan_buf, flags: int = 0, stream=None) -> None:
    """moonep_plan with options: PLAN_BOUNDED, PLAN_FOUR_LAUNCH, PLAN_TWO_LAUNCH."""
    torch = _torch()
    lay = moonep_plan_layout(dims)
    ids = _ptr(topk_ids, "topk_ids", torch.int32, 4 * dims.R * dims.S * dims.K)
    pb = _ptr(plan_buf, "plan_buf", None, lay.bytes)
    _check(_lib.moonep_plan_ex(ctypes.byref(dims), ids, pb, int(flags), _stream(stream, plan_buf)),
           "moonep_plan_ex")


def moonep_plan_noscratch(dims: Dims, topk_ids, plan_buf, bounded: bool = False,
                          stream=None) -> None:
    """moonep_plan (or moonep_plan_bounded) with the plan kernels' scratch in the
    library's static device array: plan_buf needs only persist_bytes bytes."""
    torch = _torch()
    lay = moonep_plan_layout(dims)
    ids = _ptr(topk_ids, "topk_ids", torch.int32, 4 * dims.R * dims.S * dims.K)
    pb = _ptr(plan_buf, "plan_buf", None, lay.persist_bytes)
    _check(_lib.moonep_plan_noscratch(ctypes.byref(dims), ids, pb, 1 if bounded else 0,
                                      _stream(stream, plan_buf)), "moonep_plan_noscratch")


def moonep_dispatch(dims: Dims, plan_buf, hidden, recv, stream=None) -> None:
    dt = _row_dtype(dims)
    row = dims.H * (2 if dims.dtype == BF16 else 4)
    lay = moonep_plan_layout(dims)
    _check(_lib.moonep_dispatch(
        ctypes.byref(dims), _ptr(plan_buf, "plan_buf", None, lay.persist_bytes),
        _ptr(hidden, "hidden", dt, dims.R * dims.S * row),
        _ptr(recv, "recv", dt, dims.R * dims.S * dims.K * row),
        _stream(stream, recv)), "moonep_dispatch")


def moonep_replicate(dims: Dims, plan_buf, expert_w, dup_w, block_bytes: int, stream=None) -> None:
    lay = moonep_plan_layout(dims)
    _check(_lib.moonep_replicate(
        ctypes.byref(dims), _ptr(plan_buf, "plan_buf", None, lay.persist_bytes),
        _ptr(expert_w, "expert_w", None, dims.E * block_bytes),
        _ptr(dup_w, "dup_w", None, dims.R * dims.B * block_bytes),
        int(block_bytes), _stream(stream, dup_w)), "moonep_replicate")


def moonep_combine(dims: Dims, plan_buf, y, topk_w, out, out_dtype: Optional[int] = None,
                   stream=None) -> None:
    torch = _torch()
    od = dims.dtype if out_dtype is None else int(out_dtype)
    row = dims.H * (2 if dims.dtype == BF16 else 4)
    orow = dims.H * (2 if od == BF16 else 4)
    lay = moonep_plan_layout(dims)
    _check(_lib.moonep_combine(
        ctypes.byref(dims), _ptr(plan_buf, "plan_buf", None, lay.persist_bytes),
        _ptr(y, "y", _row_dtype(dims), dims.R * dims.S * dims.K * row),
        _ptr(topk_w, "topk_w", torch.float32, 4 * dims.R * dims.S * dims.K),
        _ptr(out, "out", torch.bfloat16 if od == BF16 else torch.float32, dims.R * dims.S * orow),
        od, _stream(stream, out)), "moonep_combine")


def moonep_reduce_dup_grads(dims: Dims, plan_buf, dup_grads, home_grads, block_elems: int,
                            stream=None) -> None:
    torch = _torch()
    lay = moonep_plan_layout(dims)
    _check(_lib.moonep_reduce_dup_grads(
        ctypes.byref(dims), _ptr(plan_buf, "plan_buf", None, lay.persist_bytes),
        _ptr(dup_grads, "dup_grads", torch.float32, 4 * dims.R * dims.B * block_elems),
        _ptr(home_grads, "home_grads", torch.float32, 4 * dims.E * block_elems),
        int(block_elems), _stream(stream, home_grads)), "moonep_reduce_dup_grads")


def moonep_combine_backward(dims: Dims, plan_buf, grad_out, topk_w, y, grad_y, grad_w,
                            stream=None) -> None:
    """grad_out's dtype (float32 or bfloat16) is passed as gout_dtype; grad_y or
    grad_w may be None to skip that output (then topk_w or y may be None)."""
    torch = _torch()
    g_dt = BF16 if grad_out.dtype == torch.bfloat16 else F32
    grow = dims.H * (2 if g_dt == BF16 else 4)
    row = dims.H * (2 if dims.dtype == BF16 else 4)
    n_ent = dims.R * dims.S * dims.K
    lay = moonep_plan_layout(dims)
    ref = grad_y if grad_y is not None else grad_out
    _check(_lib.moonep_combine_backward(
        ctypes.byref(dims), _ptr(plan_buf, "plan_buf", None, lay.persist_bytes),
        _ptr(grad_out, "grad_out", None, dims.R * dims.S * grow), g_dt,
        None if grad_y is None else _ptr(topk_w, "topk_w", torch.float32, 4 * n_ent),
        None if grad_w is None else _ptr(y, "y", _row_dtype(dims), n_ent * row),
        None if grad_y is None else _ptr(grad_y, "grad_y", _row_dtype(dims), n_ent * row),
        None if grad_w is None else _ptr(grad_w, "grad_w", torch.float32, 4 * n_ent),
        _stream(stream, ref)), "moonep_combine_backward")


def moonep_dispatch_backward(dims: Dims, plan_buf, grad_recv, grad_hidden,
                             out_dtype: Optional[int] = None, stream=None) -> None:
    torch = _torch()
    od = dims.dtype if out_dtype is None else int(out_dtype)
    row = dims.H * (2 if dims.dtype == BF16 else 4)
    orow = dims.H * (2 if od == BF16 else 4)
    lay = moonep_plan_layout(dims)
    _check(_lib.moonep_dispatch_backward(
        ctypes.byref(dims), _ptr(plan_buf, "plan_buf", None, lay.persist_bytes),
        _ptr(grad_recv, "grad_recv", _row_dtype(dims), dims.R * dims.S * dims.K * row),
        _ptr(grad_hidden, "grad_hidden", torch.bfloat16 if od == BF16 else torch.float32,
             dims.R * dims.S * orow), od, _stream(stream, grad_hidden)), "moonep_dispatch_backward")


# ------------------------------------------------- the experts' products

def _tensor(t, name: str, dtype, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _dense(t, name: str, dtype, shape, device) -> int:
    """Pointer of a contiguous tensor of this dtype, shape and device."""
    if (isinstance(t, _torch().Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return t.data_ptr()
    _tensor(t, name, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _blocks(t, name: str, dtype, lead, tail, device):
    """Pointer of a tensor of lead + tail whose last dims are dense and whose leading
    dims step by one block, and that block's elements (None where no dim tells)."""
    _tensor(t, name, dtype, device)
    if t.shape != lead + tail:
        raise ValueError(f"{name} must be {lead + tail}, got {tuple(t.shape)}")
    step = 1
    for n in tail:
        step *= n
    block, seen = None, 1
    if t.is_contiguous():
        for n in lead:
            if n != 1:
                block = step
        return t.data_ptr(), block
    strides = t.stride()
    inner = 1
    for n, s in zip(reversed(tail), reversed(strides[len(lead):])):
        if n > 1 and s != inner:
            raise ValueError(f"{name}: each expert's part must be contiguous")
        inner *= n
    for n, s in zip(reversed(lead), reversed(strides[:len(lead)])):
        if n > 1 and t.numel() > 0:
            if s % seen or s // seen < step or (block is not None and s // seen != block):
                raise ValueError(f"{name}: experts must lie at equal distances")
            block = s // seen
        seen *= n
    return t.data_ptr(), block


def _pair(dims: Dims, home, dup, names, dtype, tail, device):
    """Pointers of the [E, *tail] and [R, B, *tail] tensors (dup: None with B = 0) and
    the block they share."""
    hp, hb = _blocks(home, names[0], dtype, (dims.E,), tail, device)
    dp, db = None, None
    if dims.B > 0 or dup is not None:
        dp, db = _blocks(dup, names[1], dtype, (dims.R, dims.B), tail, device)
        if dims.B == 0:
            db = None
    if hb is not None and db is not None and hb != db:
        raise ValueError(f"{names[0]} and {names[1]} must have equal distances between experts")
    if hb is None:
        hb = db
    if hb is None:
        hb = 1
        for n in tail:
            hb *= n
    return hp, dp, hb


def _gpu_of(t, name: str):
    """The device of t, which has to be a GPU."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _enqueue(device, stream, where: str, call, *args) -> None:
    """call(*args, stream) with `device` current (launches go to the current device)."""
    torch = _torch()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        rc = call(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = call(*args, handle)
    _check(rc, where)


def _seg_ptr(dims: Dims, t, device) -> int:
    G = dims.E // max(1, dims.R)
    dcap = max(1, min(dims.S * dims.K, dims.E - G))
    return _dense(t, "seg_ptr", _torch().int32, (dims.R, G + dcap + 1), device)


def _cols(t, name: str) -> int:
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) < 1:
        raise ValueError(f"{name} must have rows")
    return shape[-1]


def moonep_expert_matmul(dims: Dims, seg_ptr, x, w, dup_w, y, transposed: bool = False,
                         stream=None) -> None:
    """y [R, S*K, out] = x [R, S*K, in] times each segment's matrix: w [E, in, out] and
    dup_w [R, B, in, out] (transposed: [.., out, in]). w and dup_w may be views of larger
    blocks (w[:, 0] of an [E, 3, in, out] tensor). seg_ptr: plan_views()["seg_ptr"]."""
    dev, dt = _gpu_of(y, "y"), _row_dtype(dims)
    n_in, n_out, SK = _cols(x, "x"), _cols(y, "y"), dims.S * dims.K
    wp, dp, block = _pair(dims, w, dup_w, ("w", "dup_w"), dt,
                          (n_out, n_in) if transposed else (n_in, n_out), dev)
    _enqueue(dev, stream, "moonep_expert_matmul", _lib.moonep_expert_matmul, ctypes.byref(dims),
             _seg_ptr(dims, seg_ptr, dev), _dense(x, "x", dt, (dims.R, SK, n_in), dev), wp, dp,
             _dense(y, "y", dt, (dims.R, SK, n_out), dev), n_in, n_out, block,
             1 if transposed else 0)


def moonep_expert_matmul_wgrad(dims: Dims, seg_ptr, x, grad_y, home_grads, dup_grads,
                               transposed: bool = False, stream=None) -> None:
    """home_grads [E, in, out] and dup_grads [R, B, in, out], float32 (transposed:
    [.., out, in]): the gradients of moonep_expert_matmul's w and dup_w."""
    dev, dt = _gpu_of(home_grads, "home_grads"), _row_dtype(dims)
    n_in, n_out, SK = _cols(x, "x"), _cols(grad_y, "grad_y"), dims.S * dims.K
    hp, dp, block = _pair(dims, home_grads, dup_grads, ("home_grads", "dup_grads"),
                          _torch().float32, (n_out, n_in) if transposed else (n_in, n_out), dev)
    _enqueue(dev, stream, "moonep_expert_matmul_wgrad", _lib.moonep_expert_matmul_wgrad,
             ctypes.byref(dims), _seg_ptr(dims, seg_ptr, dev),
             _dense(x, "x", dt, (dims.R, SK, n_in), dev),
             _dense(grad_y, "grad_y", dt, (dims.R, SK, n_out), dev), hp, dp, n_in, n_out, block,
             1 if transposed else 0)


def moonep_quantize_rows(x, q, scale, stream=None) -> None:
    """q int8 [..., cols] and scale float32 [...] of the rows of x (float32 or bfloat16)."""
    torch = _torch()
    dt = getattr(x, "dtype", None)
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"x must be a float32 or bfloat16 tensor, got {dt}")
    dev, shape = _gpu_of(q, "q"), tuple(x.shape)
    cols = _cols(x, "x")
    _enqueue(dev, stream, "moonep_quantize_rows", _lib.moonep_quantize_rows,
             x.numel() // max(1, cols), cols, _dense(x, "x", dt, shape, dev),
             BF16 if dt == torch.bfloat16 else F32, _dense(q, "q", torch.int8, shape, dev),
             _dense(scale, "scale", torch.float32, shape[:-1], dev))


def moonep_expert_matmul_quant(dims: Dims, seg_ptr, x, x_scale, w, w_scale, dup_w, dup_w_scale, y,
                               stream=None) -> None:
    """y [R, S*K, out] of dims.dtype = x int8 [R, S*K, in] with x_scale [R, S*K], times
    w int8 [E, out, in] with w_scale [E, out] (dup_w [R, B, out, in], dup_w_scale [R, B, out])."""
    torch = _torch()
    dev = _gpu_of(y, "y")
    n_in, n_out, SK = _cols(x, "x"), _cols(y, "y"), dims.S * dims.K
    wp, dp, block = _pair(dims, w, dup_w, ("w", "dup_w"), torch.int8, (n_out, n_in), dev)
    sp, dsp, sblock = _pair(dims, w_scale, dup_w_scale, ("w_scale", "dup_w_scale"), torch.float32,
                            (n_out,), dev)
    _enqueue(dev, stream, "moonep_expert_matmul_quant", _lib.moonep_expert_matmul_quant,
             ctypes.byref(dims), _seg_ptr(dims, seg_ptr, dev),
             _dense(x, "x", torch.int8, (dims.R, SK, n_in), dev),
             _dense(x_scale, "x_scale", torch.float32, (dims.R, SK), dev), wp, sp, dp, dsp,
             _dense(y, "y", _row_dtype(dims), (dims.R, SK, n_out), dev), n_in, n_out, block, sblock)


# ------------------------------------------------------ norm and clipping

_DTYPE = operator.attrgetter("dtype")
_NBYTES = operator.attrgetter("nbytes")
_SHIFT = (2, 1)  # of an element's bytes: F32, BF16


class GradList:
    """Gradient tensors (float32 or bfloat16, contiguous, one device) and where their
    clipped values go (outs; default: in place), laid out for moonep_grad_sumsq and
    moonep_grad_clip. It keeps the tensors and may be used again while they live: a call
    reads their addresses and sizes anew, and one that finds others than before checks and
    lays out the list again (t.data = ..., resize_). Dtypes and strides must stay."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients, {len(self.outs)} outs")
        self._lay_out()

    def _lay_out(self) -> None:
        torch = _torch()
        n = len(self.grads)
        Tensor, codes = torch.Tensor, {torch.float32: F32, torch.bfloat16: BF16}
        device, kinds = self.grads[0].device if n and isinstance(self.grads[0], Tensor) else None, []
        # whole lists at a time: a model has hundreds of gradients
        for what, ts in (("gradient", self.grads), ("out", self.outs)):
            if ts is self.grads and kinds:
                break
            for kind in set(map(type, ts)):
                if not issubclass(kind, Tensor):
                    raise TypeError(f"every {what} must be a torch.Tensor, got {kind}")
            dtypes, gpus = list(map(_DTYPE, ts)), set(map(Tensor.get_device, ts))
            for dtype in set(dtypes):
                if dtype not in codes:
                    raise TypeError(f"every {what} must be float32 or bfloat16, got {dtype}")
            if gpus and (gpus != {device.index} or device.type != "cuda"):
                raise ValueError(f"every {what} must be a GPU tensor on the device of the others")
            if not all(map(Tensor.is_contiguous, ts)):
                raise ValueError(f"every {what} must be contiguous")
            kinds.append((dtypes, list(map(_NBYTES, ts))))
        if kinds[0] != kinds[-1]:
            raise ValueError("every out must have its gradient's dtype and elements")
        sizes, to = kinds[0][1], list(map(Tensor.data_ptr, self.outs))
        if len(set(to)) < n:
            to_some = [p for p, m in zip(to, sizes) if m > 0]
            if len(set(to_some)) < len(to_some):
                raise ValueError("two gradients have one place for their clipped values")
        self.n, self.device, self._bytes, self._to = n, device, sizes, to
        self._from = to if self.outs is self.grads else list(map(Tensor.data_ptr, self.grads))
        kind = list(map(codes.__getitem__, kinds[0][0]))
        numel = map(operator.rshift, sizes, map(_SHIFT.__getitem__, kind))
        columns = [array.array("Q", to), array.array("q", numel), array.array("i", kind)]
        if self._from is not to:
            columns.append(array.array("Q", self._from))
        self._columns = columns  # the host arrays whose addresses the calls get
        self.out_ptrs, self.numel, self.dtypes = (c.buffer_info()[0] for c in columns[:3])
        self.ptrs = self.out_ptrs if self._from is to else columns[3].buffer_info()[0]

    def refresh(self, outs: bool = False) -> None:
        """Lays the list out again if a gradient (or an out) is not where it was."""
        Tensor = _torch().Tensor
        for ts, at in ((self.grads, self._from), (self.outs, self._to))[:1 + outs]:
            if list(map(Tensor.data_ptr, ts)) != at or list(map(_NBYTES, ts)) != self._bytes:
                return self._lay_out()
            if self.outs is self.grads:
                break


def new_norm_buffer(device="cuda"):
    """The device buffer acc of moonep_grad_sumsq and moonep_grad_clip."""
    torch = _torch()
    return torch.empty(NORM_DOUBLES, dtype=torch.float64, device=device)


def _grads(grads, acc, acc_bytes: int, outs: bool = False):
    """(GradList, device, pointer of acc) of a call's gradients."""
    if isinstance(grads, GradList):
        gl = grads
        gl.refresh(outs)
    else:
        gl = GradList(grads)
    p = _ptr(acc, "acc", _torch().float64, acc_bytes)
    if gl.device is not None and acc.device != gl.device:
        raise ValueError("acc must be on the gradients' device")
    return gl, acc.device, p


def moonep_grad_sumsq(grads, acc, stream=None) -> None:
    """acc[0] = the sum of squares of all gradients (tensors or a GradList) together.
    acc: float64 [NORM_DOUBLES] (new_norm_buffer)."""
    gl, dev, p = _grads(grads, acc, 8 * NORM_DOUBLES)
    _enqueue(dev, stream, "moonep_grad_sumsq", _lib.moonep_grad_sumsq, gl.n, gl.ptrs, gl.numel,
             gl.dtypes, p)


def moonep_grad_clip(grads, acc, max_norm: float, norm=None, stream=None) -> None:
    """The gradients (tensors: in place; a GradList: into its outs) scaled so that their
    norm, sqrt(acc[0]), is max_norm at most. norm: float32 [1], receives it."""
    torch = _torch()
    gl, dev, p = _grads(grads, acc, 8, True)
    if norm is not None:
        _tensor(norm, "norm", torch.float32, dev)
        if norm.numel() < 1:
            raise ValueError("norm must hold an element")
    _enqueue(dev, stream, "moonep_grad_clip", _lib.moonep_grad_clip, gl.n, gl.ptrs, gl.out_ptrs,
             gl.numel, gl.dtypes, p, float(max_norm), None if norm is None else norm.data_ptr())


# ------------------------------------------------------------- buffer helpers

def dims_of(R: int, E: int, K: int, S: int, B: int, H: int, dtype: int) -> Dims:
    return Dims(R, E, K, S, B, dtype, H)


def new_plan_buffer(dims: Dims, device="cuda", persistent_only: bool = False):
    """A device buffer of the size the plan layout asks for (persistent_only: only
    the part that outlives the plan call, enough for moonep_plan_noscratch)."""
    torch = _torch()
    lay = moonep_plan_layout(dims)
    n = lay.persist_bytes if persistent_only else lay.bytes
    return torch.empty(n, dtype=torch.uint8, device=device)


def plan_views(dims: Dims, plan_buf) -> Dict[str, "torch.Tensor"]:
    """Typed views of the public plan arrays inside plan_buf (no copies)."""
    torch = _torch()
    lay = moonep_plan_layout(dims)
    R, E, S, K = dims.R, dims.E, dims.S, dims.K
    G, NE, dcap, pcap = E // R, R * S * K, lay.dcap, lay.pcap
    shapes = {
        "status": (1,), "maxT": (1,), "T": (E,), "hoff": (E,), "L": (R,), "keep": (R,),
        "O": (R,), "D": (R,), "Opre": (R + 1,), "Dpre": (R + 1,), "dst": (NE,), "src": (NE,),
        "n_dup": (R,), "dup_expert": (R, dcap), "dup_start": (R, dcap), "dup_count": (R, dcap),
        "seg_ptr": (R, G + dcap + 1), "seg_expert": (R, G + dcap), "n_list": (1,),
        "list_expert": (pcap,), "list_rank": (pcap,), "list_b": (pcap,), "dup_ptr": (E + 1,),
    }
    out = {}
    for name, shp in shapes.items():
        off = getattr(lay, name)
        n = 1
        for s in shp:
            n *= s
        out[name] = plan_buf[off:off + 4 * n].view(torch.int32).view(shp)
    out["maxvio"] = plan_buf[lay.maxvio:lay.maxvio + 8].view(torch.float64)
    return out
