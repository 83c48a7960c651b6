"""Python binding of libmoe.so: one expert-parallel rank's share of an MoE
layer on one MI355X (owner-aligned layout, remote-first schedule, grouped
SwiGLU FFN with flagged epilogue, consumer copy, gate-weighted scale), and the
operators around it (routing, dense product, their gradients and the scale's).

Argument marshalling only: every step runs in the HIP kernels of libmoe.so.
Tensors are torch CUDA tensors (bf16 tensors may be torch.bfloat16 or
int16/uint16 views); streams are torch.cuda.Stream objects (default: the
current stream).  The functions carry the names of the C entry points in
``include/moe.h``.  Importing this package fails loudly when libmoe.so has not
been built; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from operator import index as _int
from typing import Dict, List, Optional, Sequence

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_ECAPACITY, MOE_EHIP, MOE_ETIMEOUT, MOE_EROUTING, MOE_EUNSUPPORTED = range(7)
MODE_OVERLAP, MODE_SERIAL, MODE_COPY_ONLY, MODE_COPY_ROWS = 0, 1, 2, 3
SIGNAL_TILE, SIGNAL_GROUP = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_SWIGLU = range(6)
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

HDR_FIELDS = ["error", "M", "bands", "remote_bands", "segments", "remote_segments",
              "gateup_tiles", "down_tiles", "copy_units", "received_rows", "gateup_row_tiles",
              "down_row_tiles"]


class moe_shape(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("experts_per_rank", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("tb_m", ctypes.c_int32), ("mgb", ctypes.c_int32),
                ("tokens", ctypes.POINTER(ctypes.c_int32)), ("recv_rows", ctypes.c_int64)]


class moe_sizes(ctypes.Structure):
    _fields_ = [("plan_bytes", ctypes.c_size_t), ("rows_cap", ctypes.c_int64),
                ("bands_cap", ctypes.c_int64), ("flags_count", ctypes.c_int64),
                ("recv_rows_self", ctypes.c_int64)]


_VIEW_FIELDS = ["hdr", "c", "grp_off", "m_e", "row_off", "rb", "order", "base",
                "band_expert", "band_dst", "band_src_row", "band_dst_off", "band_valid",
                "seg_first", "seg_nbands", "seg_dst", "seg_dst_off", "seg_src_row", "seg_rows",
                "seg_unit", "src_index", "pos",
                "gu_tile_row", "gu_tile_expert", "dn_tile_row", "dn_tile_expert", "grp_band",
                "sk_counters", "sk_counters_count",
                "crow_off", "grp_crow", "band_crow", "cmp_row", "cmp_src"]


class moe_plan_view(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in _VIEW_FIELDS]


class moe_combine_opts(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("consumer_cus", ctypes.c_int32),
                ("consumer_blocks", ctypes.c_int32), ("link_mbps", ctypes.c_int32),
                ("spin_timeout_ns", ctypes.c_int64), ("events", ctypes.c_void_p * 6),
                ("x_recv", ctypes.c_void_p), ("signal", ctypes.c_int32), ("pad", ctypes.c_int32)]


class moe_route_opts(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_score", ctypes.c_int32), ("scale", ctypes.c_float)]


class moe_linear_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("depth", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("pad", ctypes.c_int32), ("ld_x", ctypes.c_int64), ("ld_w", ctypes.c_int64),
                ("ld_residual", ctypes.c_int64), ("ld_pre", ctypes.c_int64), ("ld_out", ctypes.c_int64),
                ("ld_dx", ctypes.c_int64), ("ld_dw", ctypes.c_int64)]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with `python moe_expert_tile_amd/build.py` "
                          "(there is no fallback implementation)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, V = ctypes.POINTER, ctypes.c_int, ctypes.c_void_p
    sig = {
        "moe_status_string": (ctypes.c_char_p, [I]),
        "moe_query_sizes": (I, [P(moe_shape), P(moe_sizes)]),
        "moe_plan_offsets": (I, [P(moe_shape), P(moe_plan_view)]),
        "moe_plan": (I, [P(moe_shape), V, V, V, V, V]),
        "moe_expert_combine": (I, [P(moe_shape), V, V, V, V, V, V, V, ctypes.c_uint32,
                                   P(ctypes.c_void_p), P(moe_combine_opts), V]),
        "moe_expert_combine_noalloc": (I, [P(moe_shape), V, V, V, V, V, V, V, ctypes.c_uint32,
                                           P(ctypes.c_void_p), P(moe_combine_opts), V]),
        "moe_scale": (I, [P(moe_shape), V, V, V, V, V]),
        "moe_scale_backward": (I, [P(moe_shape), V, V, V, V, V, V, V]),
        "moe_route": (I, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, V, ctypes.c_int32, ctypes.c_int64, V,
                          P(moe_route_opts), V, V, V]),
        "moe_route_backward": (I, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, V, ctypes.c_int32,
                                   ctypes.c_int64, V, V, V, P(moe_route_opts), V, ctypes.c_int64, V]),
        "moe_linear_sizes": (I, [P(moe_linear_desc), P(ctypes.c_size_t), P(ctypes.c_size_t)]),
        "moe_linear": (I, [P(moe_linear_desc), V, V, V, V, V, V, V, V]),
        "moe_linear_backward": (I, [P(moe_linear_desc), V, V, V, V, V, V, V, V, V]),
        "moe_device_status": (I, [V, V]),
        "moe_device_cus": (I, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
EXPORTED = ["moe_status_string", "moe_query_sizes", "moe_plan_offsets", "moe_plan",
            "moe_expert_combine", "moe_expert_combine_noalloc", "moe_scale", "moe_device_status",
            "moe_device_cus", "moe_scale_backward", "moe_route", "moe_route_backward", "moe_linear_sizes",
            "moe_linear", "moe_linear_backward"]


def library_path() -> str:
    return _LIB_PATH


def status_string(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoEError(rc, where)


class Shape:
    """moe_shape plus the host token array it points to."""

    def __init__(self, world: int, rank: int, experts_per_rank: int, top_k: int, hidden: int,
                 ffn: int, tb_m: int, tokens: Sequence[int], recv_rows: int, mgb: int = 1):
        self.tokens = list(int(t) for t in tokens)
        self._tok = (ctypes.c_int32 * max(1, len(self.tokens)))(*self.tokens)
        self.c = moe_shape(world, rank, experts_per_rank, top_k, hidden, ffn, tb_m, mgb,
                           ctypes.cast(self._tok, ctypes.POINTER(ctypes.c_int32)), recv_rows)

    def __getattr__(self, name):
        return getattr(self.__dict__["c"], name)

    @property
    def ptr(self):
        return ctypes.byref(self.c)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# torch's raw current stream of a device: building the Stream object that
# current_stream() returns takes 2.7 us, as long as a kernel launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def moe_query_sizes(shape: Shape) -> Dict[str, int]:
    out = moe_sizes()
    _check(_lib.moe_query_sizes(shape.ptr, ctypes.byref(out)), "moe_query_sizes")
    return {f: int(getattr(out, f)) for f, _ in moe_sizes._fields_}


def moe_plan_offsets(shape: Shape) -> Dict[str, int]:
    out = moe_plan_view()
    _check(_lib.moe_plan_offsets(shape.ptr, ctypes.byref(out)), "moe_plan_offsets")
    return {f: int(getattr(out, f)) for f in _VIEW_FIELDS}


def moe_plan(shape: Shape, topk_ids, x_recv, plan_ws, x_layout, stream=None) -> None:
    _check(_lib.moe_plan(shape.ptr, _ptr(topk_ids), _ptr(x_recv), _ptr(plan_ws), _ptr(x_layout),
                         _stream(stream)), "moe_plan")


def moe_expert_combine(shape: Shape, plan_ws, x_layout, w_gate_up, w_down, h, y, flags, epoch: int,
                       recv: List, mode: int = MODE_OVERLAP, consumer_cus: int = 0,
                       consumer_blocks: int = 0, spin_timeout_ns: int = 0,
                       events: Optional[Sequence] = None, stream=None, x_recv=None,
                       noalloc: bool = False, link_mbps: int = 0, signal: int = SIGNAL_TILE) -> None:
    """x_layout=None with x_recv given: the gate/up GEMM gathers its rows from
    x_recv through the plan's src_index (the layout is never materialized).
    noalloc=True calls moe_expert_combine_noalloc (kernel scratch in the
    library's static device array instead of the plan workspace)."""
    fn = _lib.moe_expert_combine_noalloc if noalloc else _lib.moe_expert_combine
    name = "moe_expert_combine_noalloc" if noalloc else "moe_expert_combine"
    arr = (ctypes.c_void_p * max(1, len(recv)))(*[_ptr(r) for r in recv])
    opts = moe_combine_opts()
    opts.mode = mode
    opts.consumer_cus = consumer_cus
    opts.consumer_blocks = consumer_blocks
    opts.spin_timeout_ns = spin_timeout_ns
    opts.x_recv = _ptr(x_recv)
    opts.link_mbps = int(link_mbps)
    opts.signal = int(signal)
    if events is not None:
        for i, ev in enumerate(events):
            opts.events[i] = None if ev is None else int(ev.cuda_event)
    _check(fn(shape.ptr, _ptr(plan_ws), _ptr(x_layout), _ptr(w_gate_up), _ptr(w_down), _ptr(h), _ptr(y),
              _ptr(flags), int(epoch), ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)),
              ctypes.byref(opts), _stream(stream)), name)


def moe_scale(shape: Shape, plan_ws, recv_self, topk_w, out, stream=None) -> None:
    _check(_lib.moe_scale(shape.ptr, _ptr(plan_ws), _ptr(recv_self), _ptr(topk_w), _ptr(out),
                          _stream(stream)), "moe_scale")


# --- routing, the dense product and the gradients ------------------------------
# The tensors of these calls are checked here (most of them take their sizes,
# types and row pitches from them); they run on the tensors' device (on its
# current stream unless one is given).

def _invalid(where: str, what: str):
    err = MoEError(MOE_EINVAL, where)
    err.args = (f"{err.args[0]}: {what}",)
    return err


def _mismatch(where, name, t, shape, dtype, index, kind):
    on = "the CPU" if index < 0 else f"GPU {index}"
    return _invalid(where, f"{name} is a {t.dtype} tensor {tuple(t.shape)} with strides {t.stride()} on {t.device}, "
                           f"not a {kind} {dtype} one {tuple(shape)} on {on}")


def _matrix(where, name, t, shape, dtype, index) -> int:
    """Checks a matrix of that shape with unit column stride (None passes);
    returns its row pitch, 0 (packed) where no second row shows it."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise _mismatch(where, name, t, shape, dtype, index, "row-major")
    rows, cols = shape
    pitch, step = t.stride()
    if step != 1 and cols > 1 and rows > 0 or pitch < cols and rows > 1:
        raise _mismatch(where, name, t, shape, dtype, index, "row-major")
    return pitch if rows > 1 else 0


def _packed(where, name, t, shape, dtype, index) -> Optional[int]:
    """Checks a contiguous tensor (None passes); returns its address."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise _mismatch(where, name, t, shape, dtype, index, "contiguous")
    return t.data_ptr()


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _place(where, index, stream) -> None:
    """Refuses tensors that are on no GPU, and a stream of another one."""
    if index < 0:
        raise _invalid(where, "the tensors are not on a GPU")
    if stream is not None and getattr(stream, "device_index", index) != index:
        raise _invalid(where, f"the stream is on GPU {stream.device_index}, the tensors are on GPU {index}")


def _launch(where, index, stream, fn, *args) -> None:
    """fn(*args, raw stream) with GPU `index` current; raises its errors."""
    if index < 0 or stream is not None:
        _place(where, index, stream)
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, where)


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_F32 = (torch.float32,)


def _rows(where, name, t, rows, cols, dtypes, index):
    """Checks a contiguous tensor of at least that many rows (None and plain
    addresses pass); returns its address."""
    if t is None or isinstance(t, int):
        return t
    shape = t.shape
    if (t.dtype not in dtypes or len(shape) != 2 or shape[1] != cols or shape[0] < rows or t.get_device() != index or
            not t.is_contiguous()):
        raise _mismatch(where, name, t, (rows, cols), dtypes[0], index, "contiguous")
    return t.data_ptr()


def moe_scale_backward(shape: Shape, plan_ws, recv_self, topk_w, d_out, d_recv=None, d_topk_w=None,
                       stream=None) -> None:
    """Gradients of moe_scale from d_out [T_r, d]: d_recv [T_r*k, d] (bf16, as
    recv_self and d_out) and d_topk_w float32 [T_r, k]; tensors may have more
    rows, which stay as they are.  See include/moe.h."""
    where = "moe_scale_backward"
    c = shape.c
    d, k, r = c.hidden, c.top_k, c.rank
    tokens = shape.tokens
    T = tokens[r] if 0 <= r < len(tokens) else 0   # a bad shape is the library's to refuse
    index = None
    for t in (d_out, plan_ws, recv_self, topk_w, d_recv, d_topk_w):
        if isinstance(t, torch.Tensor):
            index = t.get_device()
            break
    if isinstance(plan_ws, torch.Tensor):
        if plan_ws.get_device() != index or not plan_ws.is_contiguous():
            raise _invalid(where, "plan_ws is not a contiguous tensor on the others' device")
        plan_ws = plan_ws.data_ptr()
    args = (ctypes.byref(c), plan_ws, _rows(where, "recv_self", recv_self, T * k, d, _BF16, index),
            _rows(where, "topk_w", topk_w, T, k, _F32, index), _rows(where, "d_out", d_out, T, d, _BF16, index),
            _rows(where, "d_recv", d_recv, T * k, d, _BF16, index),
            _rows(where, "d_topk_w", d_topk_w, T, k, _F32, index))
    if index is None:   # addresses alone: on the current device
        _check(_lib.moe_scale_backward(*args, _stream(stream)), where)
    else:
        _launch(where, index, stream, _lib.moe_scale_backward, *args)


# the library only reads options, so calls with the same ones share them (plain
# numbers alone are keys: a tensor would be one by its identity)
@functools.lru_cache(maxsize=256)
def _shared_route_opts(score, renorm, n_group, topk_group, group_score, scale):
    if ctypes.c_float(scale).value == 0:   # the C options' default, 1, is not what a caller who computed 0 means
        raise _invalid("moe_route_opts", "scale is 0, not finite and above 0")
    return moe_route_opts(score, renorm, n_group, topk_group, group_score, scale)


def _route_opts(score, renorm, n_group, topk_group, group_score, scale):
    return _shared_route_opts(_int(score), 1 if renorm else 0, _int(n_group), _int(topk_group), _int(group_score),
                              float(scale))


@functools.lru_cache(maxsize=4096)
def _linear_bytes(M, N, K, dtype, out_dtype, act):
    return tuple(moe_linear_sizes(moe_linear_desc(M, N, K, dtype, out_dtype, act)).values())


def _route_tensors(where, logits, topk_ids, topk_w):
    """(sizes, type, row pitch) of the logits, and the addresses of the others."""
    code = _DTYPES.get(logits.dtype)
    if code is None or logits.dim() != 2 or topk_ids.dim() != 2:
        raise _invalid(where, "logits is a [tokens, experts] tensor of bfloat16, float16 or float32, topk_ids a "
                              "[tokens, top_k] one")
    index = logits.get_device()
    T, E = shape = logits.shape
    picks = topk_ids.shape
    if picks[0] != T:
        raise _invalid(where, f"topk_ids has {picks[0]} rows, logits {T}")
    ld = _matrix(where, "logits", logits, shape, logits.dtype, index)
    return (T, E, picks[1], logits.data_ptr(), code, ld), (
        _packed(where, "topk_ids", topk_ids, picks, torch.int32, index),
        _packed(where, "topk_w", topk_w, picks, torch.float32, index)), index


def moe_route(logits, topk_ids, topk_w, bias=None, score: int = SCORE_SOFTMAX, renorm: bool = False,
              n_group: int = 1, topk_group: int = 0, group_score: int = GROUP_MAX, scale: float = 1.0,
              stream=None) -> None:
    """Router logits [T, E] -> topk_ids int32 [T, k] (what moe_plan reads) and
    topk_w float32 [T, k] (what moe_scale reads); see include/moe.h."""
    sizes, outs, index = _route_tensors("moe_route", logits, topk_ids, topk_w)
    if bias is not None:
        bias = _packed("moe_route", "bias", bias, (sizes[1],), torch.float32, index)
    _launch("moe_route", index, stream, _lib.moe_route, *sizes, bias,
            _route_opts(score, renorm, n_group, topk_group, group_score, scale), *outs)


def moe_route_backward(logits, topk_ids, topk_w, d_topk_w, d_logits, score: int = SCORE_SOFTMAX,
                       renorm: bool = False, scale: float = 1.0, stream=None) -> None:
    """d_logits [T, E] (the logits' type) from d_topk_w float32 [T, k]; logits,
    topk_ids, topk_w, score, renorm and scale as in the moe_route call."""
    where = "moe_route_backward"
    sizes, ins, index = _route_tensors(where, logits, topk_ids, topk_w)
    g = _packed(where, "d_topk_w", d_topk_w, topk_ids.shape, torch.float32, index)
    ld_d = _matrix(where, "d_logits", d_logits, logits.shape, logits.dtype, index)
    _launch(where, index, stream, _lib.moe_route_backward, *sizes, *ins, g,
            _route_opts(score, renorm, 1, 1, GROUP_MAX, scale), d_logits.data_ptr(), ld_d)


def _linear_desc(where, x, w, out, act, out_name):
    """The product's sizes with the pitches of x, w and out, its rows n, and
    the GPU."""
    dtype, out_dtype, index = x.dtype, out.dtype, x.get_device()
    if x.dim() != 2 or w.dim() != 2 or out.dim() != 2:
        raise _invalid(where, f"x, w and {out_name} are matrices")
    if dtype is not torch.bfloat16 and dtype is not torch.float16 or (
            out_dtype is not dtype and out_dtype is not torch.float32):
        raise _invalid(where, f"x is {dtype} and {out_name} {out_dtype}: bfloat16 or float16, and the same or float32")
    M, K = xs = x.shape
    N = out.shape[1]
    n = 2 * N if act == ACT_SWIGLU else N
    return moe_linear_desc(M, N, K, _DTYPES[dtype], _DTYPES[out_dtype], act, 0, _matrix(where, "x", x, xs, dtype, index),
                           _matrix(where, "w", w, (n, K), dtype, index), 0, 0,
                           _matrix(where, out_name, out, (M, N), out_dtype, index), 0, 0), n, index


def moe_linear_sizes(desc: moe_linear_desc) -> Dict[str, int]:
    fwd, bwd = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.moe_linear_sizes(ctypes.byref(desc), ctypes.byref(fwd), ctypes.byref(bwd)), "moe_linear_sizes")
    return {"forward_bytes": fwd.value, "backward_bytes": bwd.value}


def _workspace(where, ws, need, x, stream):
    """The given workspace, checked, or one from torch's allocator on the
    stream that uses it (freed to that stream, so a later call on it may have
    the same memory)."""
    if ws is not None:
        if ws.device != x.device or not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
            raise _invalid(where, f"ws is not a contiguous tensor of {need} bytes on {x.device}")
        return ws
    if need == 0:
        return None
    if stream is not None:
        _place(where, x.get_device(), stream)
        raw = _stream(stream)
        if raw != _raw_stream(x.device.index):
            own = torch.cuda.ExternalStream(raw, device=x.device) if raw else torch.cuda.default_stream(x.device)
            with torch.cuda.stream(own):
                return torch.empty(need, dtype=torch.uint8, device=x.device)
    return torch.empty(need, dtype=torch.uint8, device=x.device)


def moe_linear(x, w, out, bias=None, residual=None, pre=None, act: int = ACT_NONE, ws=None, stream=None) -> None:
    """out = act(x w^T + bias) + residual: x [M, K], w [N, K] (SWIGLU: [2N, K],
    gate rows then up rows), out [M, N] of x's type or float32; pre, if given,
    receives x w^T + bias.  ws: at least moe_linear_sizes' forward_bytes, or
    None to take it from torch's allocator; see include/moe.h."""
    where = "moe_linear"
    d, n, index = _linear_desc(where, x, w, out, act, "out")
    if residual is not None:
        d.ld_residual = _matrix(where, "residual", residual, out.shape, out.dtype, index)
        residual = residual.data_ptr()
    if pre is not None:
        d.ld_pre = _matrix(where, "pre", pre, (x.shape[0], n), x.dtype, index)
        pre = pre.data_ptr()
    if bias is not None:
        bias = _packed(where, "bias", bias, (n,), x.dtype, index)
    need = _linear_bytes(d.rows, d.cols, d.depth, d.dtype, d.out_dtype, d.act)[0]
    if ws is not None or need:
        ws = _workspace(where, ws, need, x, stream)
    _launch(where, index, stream, _lib.moe_linear, d, x.data_ptr(), w.data_ptr(), bias, residual, pre, out.data_ptr(),
            None if ws is None else ws.data_ptr())


def moe_linear_backward(x, w, d_out, dx=None, dw=None, dbias=None, pre=None, act: int = ACT_NONE, ws=None,
                        stream=None) -> None:
    """The gradients of moe_linear that are given a tensor (dx [M, K], dw like
    w, dbias [n], all of x's type) from d_out [M, N] and, under an activation,
    the forward call's pre; see include/moe.h."""
    where = "moe_linear_backward"
    d, n, index = _linear_desc(where, x, w, d_out, act, "d_out")
    dtype = x.dtype
    d.ld_pre = _matrix(where, "pre", pre, (x.shape[0], n), dtype, index)
    d.ld_dx = _matrix(where, "dx", dx, x.shape, dtype, index)
    d.ld_dw = _matrix(where, "dw", dw, w.shape, dtype, index)
    db = _packed(where, "dbias", dbias, (n,), dtype, index)
    need = _linear_bytes(d.rows, d.cols, d.depth, d.dtype, d.out_dtype, d.act)[1]
    ws = _workspace(where, ws, need, x, stream)
    _launch(where, index, stream, _lib.moe_linear_backward, d, x.data_ptr(), w.data_ptr(), _ptr(pre),
            d_out.data_ptr(), _ptr(dx), _ptr(dw), db, _ptr(ws))


def moe_device_status(plan_ws, stream=None) -> int:
    return int(_lib.moe_device_status(_ptr(plan_ws), _stream(stream)))


def moe_device_cus() -> int:
    return int(_lib.moe_device_cus())


def timing_events(n: int = 6) -> List[torch.cuda.Event]:
    """torch events with timing, already created (recorded once) so that their
    raw handles can be recorded by the library."""
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
    for e in evs:
        e.record()
    return evs


class RankShare:
    """Device buffers of one rank's share (sized with moe_query_sizes) and the
    three calls of the path.  Buffers are torch allocations; the library
    allocates nothing."""

    def __init__(self, shape: Shape, device="cuda"):
        self.shape = shape
        self.sizes = moe_query_sizes(shape)
        self.offsets = moe_plan_offsets(shape)
        s = shape.c
        dev = torch.device(device)
        rows = self.sizes["rows_cap"]
        self.plan_ws = torch.zeros(self.sizes["plan_bytes"] // 4, dtype=torch.int32, device=dev)
        self.x_layout = torch.empty((rows, s.hidden), dtype=torch.bfloat16, device=dev)
        self.h = torch.empty((rows, s.ffn), dtype=torch.bfloat16, device=dev)
        self.y = torch.empty((rows, s.hidden), dtype=torch.bfloat16, device=dev)
        self.flags = torch.zeros(max(1, self.sizes["flags_count"]), dtype=torch.int32, device=dev)
        self.epoch = 0
        self.recv = [torch.zeros((max(1, t * s.top_k), s.hidden), dtype=torch.bfloat16, device=dev)
                     for t in shape.tokens]
        self.out = torch.empty((max(1, shape.tokens[s.rank]), s.hidden), dtype=torch.bfloat16, device=dev)

    def plan(self, topk_ids, x_recv, stream=None, materialize=True):
        """materialize=False: plan metadata only (no layout X); combine must
        then be given x_recv to gather from."""
        moe_plan(self.shape, topk_ids, x_recv, self.plan_ws, self.x_layout if materialize else None, stream)

    def combine(self, w_gate_up, w_down, mode=MODE_OVERLAP, consumer_cus=0, consumer_blocks=0,
                spin_timeout_ns=0, events=None, stream=None, epoch=None, x_recv=None, link_mbps=0,
                signal=SIGNAL_TILE, noalloc=False):
        """x_recv given: gathered rows (the gate/up GEMM reads x_recv through
        src_index instead of the layout X)."""
        if epoch is None:
            epoch = self._next_epoch()
        elif mode in (MODE_OVERLAP, MODE_SERIAL):
            # a compute mode needs a fresh epoch: with one the flags already
            # hold, the consumer could copy rows before they are written
            if not 0 < epoch <= 0xFFFFFFFF or epoch <= self.epoch:
                raise ValueError(f"epoch {epoch} is not above the last one ({self.epoch})")
            self.epoch = epoch
        moe_expert_combine(self.shape, self.plan_ws, self.x_layout if x_recv is None else None, w_gate_up,
                           w_down, self.h, self.y, self.flags, epoch, self.recv, mode, consumer_cus,
                           consumer_blocks, spin_timeout_ns, events, stream, x_recv=x_recv,
                           noalloc=noalloc, link_mbps=link_mbps, signal=signal)

    def _next_epoch(self) -> int:
        """The next epoch; after 2^32 - 1 the flags and the K-split counters
        are zeroed (on the current stream) and the epochs start again at 1."""
        if self.epoch >= 0xFFFFFFFF:
            self.flags.zero_()
            o = self.offsets["sk_counters"] // 4
            self.plan_ws[o:o + 2 * self.offsets["sk_counters_count"]].zero_()
            self.epoch = 0
        self.epoch += 1
        return self.epoch

    def scale(self, topk_w_self, stream=None):
        moe_scale(self.shape, self.plan_ws, self.recv[self.shape.c.rank], topk_w_self, self.out, stream)

    def scale_backward(self, topk_w_self, d_out, d_recv=None, d_topk_w=None, stream=None):
        """The scale step's gradients: of the rank's receive buffer and of its gate weights."""
        moe_scale_backward(self.shape, self.plan_ws, self.recv[self.shape.c.rank], topk_w_self, d_out, d_recv,
                           d_topk_w, stream)

    def status(self, stream=None) -> int:
        return moe_device_status(self.plan_ws, stream)

    def header(self) -> Dict[str, int]:
        h = self.plan_ws[self.offsets["hdr"] // 4: self.offsets["hdr"] // 4 + 16].cpu().tolist()
        return {k: h[i] for i, k in enumerate(HDR_FIELDS)}

    def end_stamps(self):
        """(last producer end, last consumer end) of the down-GEMM launch, in
        ticks of the GPU's 100 MHz wall clock (header words 12-15)."""
        o = self.offsets["hdr"] // 4
        w = self.plan_ws[o + 12: o + 16].cpu().numpy().astype(np.uint32).astype(np.uint64)
        return int(w[0] | (w[1] << np.uint64(32))), int(w[2] | (w[3] << np.uint64(32)))

    def array(self, name: str, count: int):
        o = self.offsets[name] // 4
        return self.plan_ws[o:o + count].cpu().numpy()
