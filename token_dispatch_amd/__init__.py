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

import ctypes
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

def _rows(dims: Dims, t, name: str, dtype, tail) -> int:
    """Pointer of a contiguous [R, S*K, *tail] tensor."""
    shape = (dims.R, dims.S * dims.K) + tail
    ptr = _ptr(t, name, dtype)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    return ptr


def _blocks(t, name: str, dtype, lead, tail):
    """Pointer of a tensor of lead + tail whose last dims are dense and whose leading
    dims step by one block, and that block's elements (None where no dim tells)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != lead + tail:
        raise ValueError(f"{name} must be {lead + tail}, got {tuple(t.shape)}")
    step = 1
    for n, s in zip(reversed(tail), reversed(t.stride()[len(lead):])):
        if n > 1 and s != step:
            raise ValueError(f"{name}: each expert's part must be contiguous")
        step *= n
    block, seen = None, 1
    for n, s in zip(reversed(lead), reversed(t.stride()[:len(lead)])):
        if n > 1 and t.numel() > 0:
            if s % seen or s // seen < step or (block is not None and s // seen != block):
                raise ValueError(f"{name}: experts must lie at equal distances")
            block = s // seen
        seen *= n
    return t.data_ptr(), block


def _pair(dims: Dims, home, dup, names, dtype, tail):
    """Pointers of the [E, *tail] and [R, B, *tail] tensors (dup: None with B = 0) and
    the block they share."""
    hp, hb = _blocks(home, names[0], dtype, (dims.E,), tail)
    dp, db = None, None
    if dims.B > 0 or dup is not None:
        dp, db = _blocks(dup, names[1], dtype, (dims.R, dims.B), tail)
    if hb is not None and db is not None and hb != db:
        raise ValueError(f"{names[0]} and {names[1]} must have equal distances between experts")
    dense = 1
    for n in tail:
        dense *= n
    return hp, dp, hb if hb is not None else db if db is not None else dense


def _same_device(*tensors):
    """A context with the tensors' device current; refuses tensors of several."""
    torch = _torch()
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"tensors on different devices: {sorted(map(str, devs))}")
    return torch.cuda.device(devs.pop())


def _seg_ptr(dims: Dims, t) -> int:
    lay = moonep_plan_layout(dims)
    ptr = _ptr(t, "seg_ptr", _torch().int32)
    shape = (dims.R, dims.E // dims.R + lay.dcap + 1)
    if tuple(t.shape) != shape:
        raise ValueError(f"seg_ptr must be {shape}, got {tuple(t.shape)}")
    return ptr


def moonep_expert_matmul(dims: Dims, seg_ptr, x, w, dup_w, y, transposed: bool = False,
                         stream=None) -> None:
    """y [R, S*K, out] = x [R, S*K, in] times each segment's matrix: w [E, in, out] and
    dup_w [R, B, in, out] (transposed: [.., out, in]). w and dup_w may be views of larger
    blocks (w[:, 0] of an [E, 3, in, out] tensor). seg_ptr: plan_views()["seg_ptr"]."""
    dt, n_in, n_out = _row_dtype(dims), x.shape[-1], y.shape[-1]
    tail = (n_out, n_in) if transposed else (n_in, n_out)
    wp, dp, block = _pair(dims, w, dup_w, ("w", "dup_w"), dt, tail)
    with _same_device(seg_ptr, x, w, dup_w, y):
        _check(_lib.moonep_expert_matmul(
            ctypes.byref(dims), _seg_ptr(dims, seg_ptr), _rows(dims, x, "x", dt, (n_in,)), wp, dp,
            _rows(dims, y, "y", dt, (n_out,)), n_in, n_out, block, 1 if transposed else 0,
            _stream(stream, y)), "moonep_expert_matmul")


def moonep_expert_matmul_wgrad(dims: Dims, seg_ptr, x, grad_y, home_grads, dup_grads,
                               transposed: bool = False, stream=None) -> None:
    """home_grads [E, in, out] and dup_grads [R, B, in, out], float32 (transposed:
    [.., out, in]): the gradients of moonep_expert_matmul's w and dup_w."""
    torch = _torch()
    dt, n_in, n_out = _row_dtype(dims), x.shape[-1], grad_y.shape[-1]
    tail = (n_out, n_in) if transposed else (n_in, n_out)
    hp, dp, block = _pair(dims, home_grads, dup_grads, ("home_grads", "dup_grads"), torch.float32, tail)
    with _same_device(seg_ptr, x, grad_y, home_grads, dup_grads):
        _check(_lib.moonep_expert_matmul_wgrad(
            ctypes.byref(dims), _seg_ptr(dims, seg_ptr), _rows(dims, x, "x", dt, (n_in,)),
            _rows(dims, grad_y, "grad_y", dt, (n_out,)), hp, dp, n_in, n_out, block,
            1 if transposed else 0, _stream(stream, home_grads)), "moonep_expert_matmul_wgrad")


def moonep_quantize_rows(x, q, scale, stream=None) -> None:
    """q int8 [..., cols] and scale float32 [...] of the rows of x (float32 or bfloat16)."""
    torch = _torch()
    if isinstance(x, torch.Tensor) and x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    xp, qp, sp = _ptr(x, "x"), _ptr(q, "q", torch.int8), _ptr(scale, "scale", torch.float32)
    if x.dim() < 1 or q.shape != x.shape or scale.shape != x.shape[:-1]:
        raise ValueError("q must have x's shape, and scale that of its rows")
    with _same_device(x, q, scale):
        _check(_lib.moonep_quantize_rows(
            scale.numel(), x.shape[-1], xp, BF16 if x.dtype == torch.bfloat16 else F32, qp, sp,
            _stream(stream, q)), "moonep_quantize_rows")


def moonep_expert_matmul_quant(dims: Dims, seg_ptr, x, x_scale, w, w_scale, dup_w, dup_w_scale, y,
                               stream=None) -> None:
    """y [R, S*K, out] of dims.dtype = x int8 [R, S*K, in] with x_scale [R, S*K], times
    w int8 [E, out, in] with w_scale [E, out] (dup_w [R, B, out, in], dup_w_scale [R, B, out])."""
    torch = _torch()
    n_in, n_out = x.shape[-1], y.shape[-1]
    wp, dp, block = _pair(dims, w, dup_w, ("w", "dup_w"), torch.int8, (n_out, n_in))
    sp, dsp, sblock = _pair(dims, w_scale, dup_w_scale, ("w_scale", "dup_w_scale"), torch.float32,
                            (n_out,))
    with _same_device(seg_ptr, x, x_scale, w, w_scale, dup_w, dup_w_scale, y):
        _check(_lib.moonep_expert_matmul_quant(
            ctypes.byref(dims), _seg_ptr(dims, seg_ptr), _rows(dims, x, "x", torch.int8, (n_in,)),
            _rows(dims, x_scale, "x_scale", torch.float32, ()), wp, sp, dp, dsp,
            _rows(dims, y, "y", _row_dtype(dims), (n_out,)), n_in, n_out, block, sblock,
            _stream(stream, y)), "moonep_expert_matmul_quant")


# ------------------------------------------------------ norm and clipping

class GradList:
    """Gradient tensors (float32 or bfloat16, contiguous, one device) and where their
    clipped values go (outs; default: in place), laid out for moonep_grad_sumsq and
    moonep_grad_clip. It keeps the tensors and may be used again while they live."""

    def __init__(self, grads, outs=None):
        torch = _torch()
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients, {len(self.outs)} outs")
        codes = {torch.float32: F32, torch.bfloat16: BF16}
        self.device = None
        for what, ts in (("gradient", self.grads), ("out", self.outs)):
            for i, t in enumerate(ts):
                if not isinstance(t, torch.Tensor):
                    raise TypeError(f"{what} {i} must be a torch.Tensor")
                if self.device is None:
                    self.device = t.device
                if t.device.type != "cuda" or t.device != self.device:
                    raise ValueError(f"{what} {i} must be a GPU tensor on the device of the others")
                if not t.is_contiguous():
                    raise ValueError(f"{what} {i} must be contiguous")
                if t.dtype not in codes:
                    raise TypeError(f"{what} {i} must be float32 or bfloat16, got {t.dtype}")
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if g.dtype != o.dtype or g.numel() != o.numel():
                raise ValueError(f"out {i} must have its gradient's dtype and elements")
        n = self.n = len(self.grads)
        self.ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.grads])
        self.out_ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.outs])
        self.numel = (ctypes.c_int64 * n)(*[t.numel() for t in self.grads])
        self.dtypes = (ctypes.c_int32 * n)(*[codes[t.dtype] for t in self.grads])


def _grad_list(grads) -> GradList:
    return grads if isinstance(grads, GradList) else GradList(grads)


def _acc(acc, gl: GradList) -> int:
    torch = _torch()
    p = _ptr(acc, "acc", torch.float64, 8 * NORM_DOUBLES)
    if gl.device is not None and acc.device != gl.device:
        raise ValueError("acc must be on the gradients' device")
    return p


def new_norm_buffer(device="cuda"):
    """The device buffer acc of moonep_grad_sumsq and moonep_grad_clip."""
    torch = _torch()
    return torch.empty(NORM_DOUBLES, dtype=torch.float64, device=device)


def moonep_grad_sumsq(grads, acc, stream=None) -> None:
    """acc[0] = the sum of squares of all gradients (tensors or a GradList) together."""
    gl = _grad_list(grads)
    p = _acc(acc, gl)
    with _same_device(acc):
        _check(_lib.moonep_grad_sumsq(gl.n, gl.ptrs, gl.numel, gl.dtypes, p, _stream(stream, acc)),
               "moonep_grad_sumsq")


def moonep_grad_clip(grads, acc, max_norm: float, norm=None, stream=None) -> None:
    """The gradients (tensors: in place; a GradList: into its outs) scaled so that their
    norm, sqrt(acc[0]), is max_norm at most. norm: float32 [1], receives it."""
    torch = _torch()
    gl = _grad_list(grads)
    p = _acc(acc, gl)
    with _same_device(acc, norm):
        _check(_lib.moonep_grad_clip(
            gl.n, gl.ptrs, gl.out_ptrs, gl.numel, gl.dtypes, p, float(max_norm),
            None if norm is None else _ptr(norm, "norm", torch.float32, 4), _stream(stream, acc)),
            "moonep_grad_clip")


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
