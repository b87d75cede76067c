"""ctypes binding of libspc.so (the C ABI declared in include/spc.h).

Each ``spc_*`` function here has the name of the C entry point it calls and
only marshals arguments: it takes torch CUDA tensors, allocates the outputs and
workspace with torch (device memory only), passes raw pointers and the current
CUDA stream, and checks the returned status.  Every computation runs in the
library's CUDA kernels; there is no CPU fallback.  If libspc.so has not been
built, loading raises ``SpcLibraryMissing``.
"""

from __future__ import annotations

import ctypes
import functools
import operator
import os
import threading
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libspc.so")

SPC_OK = 0
SPC_ERR_INVALID_ARG = 1
STATUS_NAMES = {
    0: "SPC_OK", 1: "SPC_ERR_INVALID_ARG", 2: "SPC_ERR_COORD_RANGE", 3: "SPC_ERR_DUPLICATE",
    4: "SPC_ERR_TABLE_FULL", 5: "SPC_ERR_CAPACITY", 6: "SPC_ERR_UNSUPPORTED", 7: "SPC_ERR_CUDA",
    8: "SPC_ERR_WORKSPACE", 9: "SPC_ERR_TIMEOUT", 10: "SPC_ERR_ROW_INDEX",
}
SPC_F32, SPC_F16, SPC_BF16 = 0, 1, 2
SPC_PREC_EXACT, SPC_PREC_TF32 = 0, 1
SPC_MAP_TRANSPOSED, SPC_MAP_SUBM_MIRROR = 0, 1
SPC_SCORE_SOFTMAX, SPC_SCORE_SIGMOID = 0, 1
SPC_MAX_TOP_K = 32

_DTYPES = {torch.float32: SPC_F32, torch.float16: SPC_F16, torch.bfloat16: SPC_BF16}


class SpcLibraryMissing(RuntimeError):
    pass


class SpcError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class Geom(ctypes.Structure):
    _fields_ = [("ksize", ctypes.c_int32 * 3), ("stride", ctypes.c_int32 * 3),
                ("pad", ctypes.c_int32 * 3), ("dil", ctypes.c_int32 * 3)]


def _triple(v) -> tuple:
    if isinstance(v, int):
        return (v, v, v)
    t = tuple(int(a) for a in v)
    assert len(t) == 3
    return t


def make_geom(ksize=3, stride=1, pad=0, dil=1) -> Geom:
    g = Geom()
    for name, v in (("ksize", ksize), ("stride", stride), ("pad", pad), ("dil", dil)):
        arr = getattr(g, name)
        for a, x in enumerate(_triple(v)):
            arr[a] = x
    return g


_lock = threading.Lock()
_lib = None

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t
_I3 = ctypes.c_int32 * 3
_GP = ctypes.POINTER(Geom)


def lib():
    """The loaded libspc.so (raises SpcLibraryMissing if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise SpcLibraryMissing(
                    f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                    "(there is no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            L.spc_status_string.argtypes = [_i32]
            L.spc_status_string.restype = ctypes.c_char_p
            L.spc_version.argtypes = []
            L.spc_version.restype = _i32
            L.spc_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.spc_set_wait_limit_ns.restype = _i32
            L.spc_get_wait_limit_ns.argtypes = []
            L.spc_get_wait_limit_ns.restype = ctypes.c_uint64
            L.spc_out_shape.argtypes = [_I3, _GP, _I3]
            L.spc_out_shape.restype = _i32
            L.spc_indice_map_workspace_size.argtypes = [_i64]
            L.spc_indice_map_workspace_size.restype = _sz
            L.spc_build_indice_map.argtypes = [_p, _i64, _i32, _I3, _GP, _i32, _p, _i64, _p, _p,
                                               _p, _p, _p, _p, _sz, _p]
            L.spc_build_indice_map.restype = _i32
            L.spc_strided_out_coords_workspace_size.argtypes = [_i64, _GP]
            L.spc_strided_out_coords_workspace_size.restype = _sz
            L.spc_strided_out_coords.argtypes = [_p, _i64, _i32, _I3, _GP, _I3, _p, _i64, _p, _p,
                                                 _p, _sz, _p]
            L.spc_strided_out_coords.restype = _i32
            L.spc_conv_workspace_size.argtypes = [_i32, _i64, _i64, _i32, _i32, _i32]
            L.spc_conv_workspace_size.restype = _sz
            L.spc_conv_fwd.argtypes = [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i32, _i32, _i32,
                                       _i32, _p, _p, _p, _sz, _p]
            L.spc_conv_fwd.restype = _i32
            L.spc_conv_fwd_fused.argtypes = [_p, _p, _p, _p, _p, _p, _i32, _i64, _i64, _i32, _i32, _i32,
                                             _i32, _p, ctypes.c_float, _i32, _p, _p, _p, _sz, _p]
            L.spc_conv_fwd_fused.restype = _i32
            L.spc_maxpool_fwd.argtypes = [_p, _p, _p, _i32, _i64, _i64, _i32, _i32, _p, _p, _p]
            L.spc_maxpool_fwd.restype = _i32
            L.spc_maxpool_dgrad.argtypes = [_p, _p, _p, _i32, _i64, _i64, _i32, _i32, _p, _p]
            L.spc_maxpool_dgrad.restype = _i32
            L.spc_conv_inverse.argtypes = [_p, _p, _p, _p, _p, _p, _i32, _i64, _i64, _i32, _i32, _i32,
                                           _i32, _p, _p, _p, _sz, _p]
            L.spc_map_row_order_workspace_size.argtypes = [_i64]
            L.spc_map_row_order_workspace_size.restype = _sz
            L.spc_map_row_order.argtypes = [_p, _i32, _i64, _p, _p, _p, _sz, _p]
            L.spc_map_row_order.restype = _i32
            L.spc_conv_inverse.restype = _i32
            L.spc_conv_int8_workspace_size.argtypes = [_i32, _i32, _i32]
            L.spc_conv_int8_workspace_size.restype = _sz
            L.spc_conv_fwd_int8.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i32, _i64, _i64, _i32, _i32,
                                            _p, ctypes.c_float, _i32, _p, _p, _p, _sz, _p]
            L.spc_conv_fwd_int8.restype = _i32
            L.spc_conv_dgrad.argtypes = [_p, _p, _p, _i32, _p, _p, _i32, _i64, _i64, _i32, _i32,
                                         _i32, _i32, _p, _p, _p, _sz, _p]
            L.spc_conv_dgrad.restype = _i32
            L.spc_conv_wgrad_workspace_size.argtypes = [_i32, _i64, _i64, _i32, _i32, _i32]
            L.spc_conv_wgrad_workspace_size.restype = _sz
            L.spc_conv_wgrad.argtypes = [_p, _p, _p, _i32, _i64, _i64, _i32, _i32, _i32, _i32,
                                         _p, _p, _p, _sz, _p]
            L.spc_conv_wgrad.restype = _i32
            _f = ctypes.c_float
            L.spc_row_segments_workspace_size.argtypes = [_i64, _i32]
            L.spc_row_segments_workspace_size.restype = _sz
            L.spc_row_segments.argtypes = [_p, _i64, _i64, _i32, _p, _p, _p, _sz, _p]
            L.spc_row_segments.restype = _i32
            L.spc_group_norm_workspace_size.argtypes = [_i64, _i32, _i32, _i32, _i32]
            L.spc_group_norm_workspace_size.restype = _sz
            L.spc_group_norm_fwd.argtypes = [_p, _p, _p, _p, _p, _i32, _i64, _i32, _i32, _f, _i32, _i32,
                                             _p, _p, _p, _p, _p, _sz, _p]
            L.spc_group_norm_fwd.restype = _i32
            L.spc_group_norm_bwd.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i32, _i64, _i32, _i32, _i32,
                                             _i32, _p, _p, _p, _p, _p, _sz, _p]
            L.spc_group_norm_bwd.restype = _i32
            L.spc_dropout_fwd.argtypes = [_p, _p, _i64, ctypes.c_double, _p, _i32, _p, _p]
            L.spc_dropout_fwd.restype = _i32
            L.spc_dropout_bwd.argtypes = [_p, _i64, ctypes.c_double, _p, _i32, _p, _p]
            L.spc_dropout_bwd.restype = _i32
            L.spc_grouped_workspace_size.argtypes = [_i32, _i64, _i32, _i32, _i32, _i32]
            L.spc_grouped_workspace_size.restype = _sz
            for f in (L.spc_grouped_fwd, L.spc_grouped_dgrad):
                f.argtypes = [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i32, _i32, _i32, _p, _p, _p, _sz, _p]
                f.restype = _i32
            L.spc_grouped_wgrad.argtypes = [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _i32, _i32, _i32,
                                            _p, _p, _p, _sz, _p]
            L.spc_grouped_wgrad.restype = _i32
            L.spc_layer_norm_workspace_size.argtypes = [_i64, _i32]
            L.spc_layer_norm_workspace_size.restype = _sz
            L.spc_layer_norm_fwd.argtypes = [_p, _p, _p, _i64, _i32, _f, _i32, _p, _p, _p, _p]
            L.spc_layer_norm_bwd.argtypes = [_p, _p, _p, _p, _p, _i64, _i32, _i32, _p, _p, _p, _p, _sz, _p]
            L.spc_rope_steps.argtypes = [_I3, ctypes.c_double, _p]
            L.spc_rope_fwd.argtypes = [_p, _i64, _p, _I3, _p, _i64, _i32, _i32, _i32, _p, _i64, _p]
            L.spc_rope_bwd.argtypes = L.spc_rope_fwd.argtypes
            L.spc_route_fwd.argtypes = [_p, _p, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _f, _i32, _p, _p, _p]
            L.spc_route_bwd.argtypes = [_p, _p, _p, _i64, _i32, _i32, _i32, _i32, _f, _i32, _p, _p, _p]
            L.spc_attention_workspace_size.argtypes = [_i64, _i64, _i32, _i32, _i32, _i32, _i32, _i32]
            L.spc_attention_workspace_size.restype = _sz
            L.spc_attention_fwd.argtypes = [_p, _i64, _p, _i64, _p, _i64, _p, _p, _i32, _i64, _i64, _i32, _i32, _i32,
                                            _f, _i32, _p, _i64, _p, _p, _p, _sz, _p]
            L.spc_attention_bwd.argtypes = [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i32, _i64,
                                            _i64, _i32, _i32, _i32, _f, _i32, _p, _i64, _p, _i64, _p, _i64, _p, _p,
                                            _sz, _p]
            for f in (L.spc_layer_norm_fwd, L.spc_layer_norm_bwd, L.spc_rope_steps, L.spc_rope_fwd, L.spc_rope_bwd,
                      L.spc_route_fwd, L.spc_route_bwd, L.spc_attention_fwd, L.spc_attention_bwd):
                f.restype = _i32
            _lib = L
    return _lib


def _check(code: int, where: str):
    if code != SPC_OK:
        raise SpcError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    # the raw handle, without the Stream object that torch.cuda.current_stream builds around it
    return torch._C._cuda_getCurrentRawStream(device.index)


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t if t.is_contiguous() else t.contiguous()


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def new_status(device) -> torch.Tensor:
    """A zeroed device status word (sticky error flag of the data-dependent checks)."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def check_status(status: torch.Tensor, where: str = "spc"):
    """Synchronise on the status word and raise SpcError if a kernel reported an error."""
    code = int(status.item())
    if code != SPC_OK:
        raise SpcError(code, where)


def spc_status_string(code: int) -> str:
    return lib().spc_status_string(code).decode()


def spc_version() -> int:
    return int(lib().spc_version())


def spc_set_wait_limit_ns(ns: int) -> None:
    """Bound (ns) of the waits of one warp role on another in the pipelined
    tensor-core kernels launched afterwards (a wait that runs out sets
    SPC_ERR_TIMEOUT in the call's status word)."""
    _check(lib().spc_set_wait_limit_ns(int(ns)), "spc_set_wait_limit_ns")


def spc_get_wait_limit_ns() -> int:
    return int(lib().spc_get_wait_limit_ns())


def spc_out_shape(in_shape, ksize=3, stride=2, pad=1, dil=1) -> tuple:
    g = make_geom(ksize, stride, pad, dil)
    out = _I3()
    _check(lib().spc_out_shape(_I3(*_triple(in_shape)), ctypes.byref(g), out), "spc_out_shape")
    return tuple(out)


def spc_indice_map_workspace_size(n_in: int) -> int:
    return int(lib().spc_indice_map_workspace_size(n_in))


def spc_build_indice_map(coords: torch.Tensor, batch: int, in_shape: Sequence[int], ksize=3,
                         stride=1, pad=0, dil=1, subm: bool = True,
                         out_coords: Optional[torch.Tensor] = None, with_transpose: bool = False,
                         with_mask: bool = True, status: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Indice map [K, N_out] (+ transpose [K, N_in], pair counts [K], row masks [N_out]).

    Returns a dict with keys imap, imap_t (or None), pair_count, mask (or None),
    status, ws.  Data errors land in `status`; call check_status() to raise them.
    Passing the dict of an earlier call as `out` reuses its buffers (no
    allocation, so the call can be captured in a CUDA graph).
    """
    coords = _cuda(coords, "coords").to(torch.int32)
    dev = coords.device
    n_in = coords.shape[0]
    g = make_geom(ksize, stride, pad, dil)
    K = g.ksize[0] * g.ksize[1] * g.ksize[2]
    if subm:
        n_out = n_in
        oc = None
    else:
        oc = _cuda(out_coords, "out_coords").to(torch.int32)
        n_out = oc.shape[0]
    if out is not None:
        imap, imap_t, pair_count, mask = out["imap"], out["imap_t"], out["pair_count"], out["mask"]
        status = out["status"] if status is None else status
        ws = out["ws"] if ws is None else ws
    else:
        imap = torch.empty((K, n_out), dtype=torch.int32, device=dev)
        imap_t = (torch.empty((K, n_in), dtype=torch.int32, device=dev)
                  if (with_transpose and not subm) else None)
        pair_count = torch.empty(K, dtype=torch.int32, device=dev)
        mask = torch.empty(n_out, dtype=torch.int32, device=dev) if (with_mask and K <= 32) else None
    status = new_status(dev) if status is None else status
    nbytes = spc_indice_map_workspace_size(n_in)
    if ws is None or ws.numel() < nbytes:
        ws = _workspace(nbytes, dev)
    code = lib().spc_build_indice_map(
        _ptr(coords), n_in, batch, _I3(*_triple(in_shape)), ctypes.byref(g), 1 if subm else 0,
        _ptr(oc), n_out, _ptr(imap), _ptr(imap_t), _ptr(pair_count), _ptr(mask), _ptr(status),
        _ptr(ws), ws.numel(), _stream(dev))
    _check(code, "spc_build_indice_map")
    return dict(imap=imap, imap_t=imap_t, pair_count=pair_count, mask=mask, status=status, ws=ws)


def spc_strided_out_coords(coords: torch.Tensor, batch: int, in_shape, ksize=3, stride=2, pad=1,
                           dil=1, cap: Optional[int] = None, status: Optional[torch.Tensor] = None):
    """Output coordinate set [N_out, 4] (sorted by (b, z, y, x)) and the output grid.

    Reads N_out back to the host (one synchronisation) to trim the buffer.
    """
    coords = _cuda(coords, "coords").to(torch.int32)
    dev = coords.device
    n_in = coords.shape[0]
    g = make_geom(ksize, stride, pad, dil)
    K = g.ksize[0] * g.ksize[1] * g.ksize[2]
    cap = n_in * K if cap is None else int(cap)
    out = torch.empty((max(cap, 1), 4), dtype=torch.int32, device=dev)
    n_out = torch.zeros(1, dtype=torch.int64, device=dev)
    status = new_status(dev) if status is None else status
    nbytes = int(lib().spc_strided_out_coords_workspace_size(n_in, ctypes.byref(g)))
    ws = _workspace(nbytes, dev)
    out_shape = _I3()
    code = lib().spc_strided_out_coords(
        _ptr(coords), n_in, batch, _I3(*_triple(in_shape)), ctypes.byref(g), out_shape, _ptr(out),
        cap, _ptr(n_out), _ptr(status), _ptr(ws), ws.numel(), _stream(dev))
    _check(code, "spc_strided_out_coords")
    n = int(n_out.item())
    check_status(status, "spc_strided_out_coords")
    return out[:n], tuple(out_shape)


def spc_conv_fwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor],
                 imap: Optional[torch.Tensor], mask: Optional[torch.Tensor] = None,
                 n_out: Optional[int] = None, precision: int = SPC_PREC_EXACT,
                 out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[o] = bias + sum over pairs of x[imap[k, o]] W[k]; y has x's dtype.

    Pass `out`, `ws` (spc_conv_workspace_size bytes) and `status` to call
    without allocating (e.g. inside CUDA-graph capture).  `perm` (with its
    `mask`) from spc_map_row_order(imap) computes the tiles in that row order
    (through spc_conv_fwd_fused, which takes it)."""
    if perm is not None:
        return spc_conv_fwd_fused(x, w, bias, imap, mask, n_out=n_out, precision=precision,
                                  out=out, status=status, ws=ws, perm=perm)
    x = _cuda(x, "x")
    w = _cuda(w, "w").to(x.dtype)
    b = _cuda(bias, "bias").to(x.dtype) if bias is not None else None
    K, cin, cout = w.shape
    if imap is not None:
        imap = _cuda(imap, "imap")
        n_out = imap.shape[1]
    elif n_out is None:
        n_out = x.shape[0]
    y = torch.empty((n_out, cout), dtype=x.dtype, device=x.device) if out is None else out
    dt = _DTYPES[x.dtype]
    nbytes = int(lib().spc_conv_workspace_size(K, x.shape[0], n_out, cin, cout, dt))
    if nbytes and (ws is None or ws.numel() < nbytes):
        ws = _workspace(nbytes, x.device)
    code = lib().spc_conv_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(imap), _ptr(mask), K, x.shape[0],
                              n_out, cin, cout, dt, precision, _ptr(y), _ptr(status), _ptr(ws),
                              0 if ws is None else ws.numel(), _stream(x.device))
    _check(code, "spc_conv_fwd")
    return y


SPC_ACT_NONE, SPC_ACT_RELU, SPC_ACT_SILU = 0, 1, 2


def spc_conv_fwd_fused(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor],
                       imap: Optional[torch.Tensor], mask: Optional[torch.Tensor] = None,
                       residual: Optional[torch.Tensor] = None, add_scale: float = 1.0,
                       act: int = SPC_ACT_NONE, n_out: Optional[int] = None,
                       precision: int = SPC_PREC_EXACT, out: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None,
                       perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[o] = act(bias + sum over pairs of x[imap[k, o]] W[k] + add_scale residual[o]);
    `perm` (with its `mask`) from spc_map_row_order(imap) groups the tiles' rows."""
    x = _cuda(x, "x")
    w = _cuda(w, "w").to(x.dtype)
    b = _cuda(bias, "bias").to(x.dtype) if bias is not None else None
    res = _cuda(residual, "residual").to(x.dtype) if residual is not None else None
    K, cin, cout = w.shape
    if imap is not None:
        imap = _cuda(imap, "imap")
        n_out = imap.shape[1]
    elif n_out is None:
        n_out = x.shape[0]
    y = torch.empty((n_out, cout), dtype=x.dtype, device=x.device) if out is None else out
    dt = _DTYPES[x.dtype]
    nbytes = int(lib().spc_conv_workspace_size(K, x.shape[0], n_out, cin, cout, dt))
    if nbytes and (ws is None or ws.numel() < nbytes):
        ws = _workspace(nbytes, x.device)
    code = lib().spc_conv_fwd_fused(_ptr(x), _ptr(w), _ptr(b), _ptr(imap), _ptr(mask), _ptr(perm), K,
                                    x.shape[0], n_out, cin, cout, dt, precision, _ptr(res),
                                    float(add_scale), int(act), _ptr(y), _ptr(status), _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(x.device))
    _check(code, "spc_conv_fwd_fused")
    return y


def spc_maxpool_fwd(x: torch.Tensor, imap: torch.Tensor, mask: Optional[torch.Tensor] = None,
                    with_arg: bool = True, out: Optional[torch.Tensor] = None,
                    arg: Optional[torch.Tensor] = None):
    """Sparse max pool on a strided map imap [K, N_out]: returns (y [N_out, C], arg) where
    arg [N_out, C] uint8 holds the offset each channel took (None unless with_arg)."""
    x = _cuda(x, "x")
    m = _cuda(imap, "imap")
    K, n_out = m.shape
    c = x.shape[1]
    y = torch.empty((n_out, c), dtype=x.dtype, device=x.device) if out is None else out
    if with_arg and arg is None:
        arg = torch.empty((n_out, c), dtype=torch.uint8, device=x.device)
    code = lib().spc_maxpool_fwd(_ptr(x), _ptr(m), _ptr(mask), K, x.shape[0], n_out, c,
                                 _DTYPES[x.dtype], _ptr(y), _ptr(arg if with_arg else None),
                                 _stream(x.device))
    _check(code, "spc_maxpool_fwd")
    return y, (arg if with_arg else None)


def spc_maxpool_dgrad(dy: torch.Tensor, imap_t: torch.Tensor, arg: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of spc_maxpool_fwd through the transposed map imap_t [K, N_in]."""
    dy = _cuda(dy, "dy")
    mt = _cuda(imap_t, "imap_t")
    K, n_in = mt.shape
    c = dy.shape[1]
    dx = torch.empty((n_in, c), dtype=dy.dtype, device=dy.device) if out is None else out
    code = lib().spc_maxpool_dgrad(_ptr(dy), _ptr(mt), _ptr(_cuda(arg, "arg")), K, n_in,
                                   dy.shape[0], c, _DTYPES[dy.dtype], _ptr(dx), _stream(dy.device))
    _check(code, "spc_maxpool_dgrad")
    return dx


def spc_map_row_order(map_: Optional[torch.Tensor], ws: Optional[torch.Tensor] = None,
                      mask: Optional[torch.Tensor] = None, K: Optional[int] = None,
                      perm: Optional[torch.Tensor] = None):
    """(mask [n] uint32, perm [n] int32): rows of map [K, n] grouped by offset mask.

    With map_ None, `mask` (the row masks spc_build_indice_map wrote) and `K`
    are read instead of the map.  Passing `ws` and `perm` (and `mask`) avoids
    allocation (e.g. inside CUDA-graph capture)."""
    if map_ is not None:
        m = _cuda(map_, "map")
        K, n = m.shape
        dev = m.device
        mask = torch.empty(n, dtype=torch.int32, device=dev) if mask is None else mask
    else:
        m = None
        assert mask is not None and K is not None
        n, dev = mask.shape[0], mask.device
    perm = torch.empty(n, dtype=torch.int32, device=dev) if perm is None else perm
    nbytes = int(lib().spc_map_row_order_workspace_size(n))
    if ws is None or ws.numel() < nbytes:
        ws = _workspace(nbytes, dev)
    code = lib().spc_map_row_order(_ptr(m), int(K), n, _ptr(mask), _ptr(perm), _ptr(ws), ws.numel(),
                                   _stream(dev))
    _check(code, "spc_map_row_order")
    return mask, perm


def spc_conv_inverse(y: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor],
                     imap_t: torch.Tensor, precision: int = SPC_PREC_EXACT,
                     out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, mask_t: Optional[torch.Tensor] = None,
                     perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Inverse of a strided conv through its transposed map imap_t [K, N_in]:
    out[i] = bias + sum over pairs imap_t[k, i] = o of y[o] W[k]; out [N_in, Cout].
    mask_t / perm from spc_map_row_order(imap_t) let the kernel skip unused offsets."""
    y = _cuda(y, "y")
    w = _cuda(w, "w").to(y.dtype)
    b = _cuda(bias, "bias").to(y.dtype) if bias is not None else None
    m = _cuda(imap_t, "imap_t")
    K, cy, cout = w.shape
    n_out = m.shape[1]
    o = torch.empty((n_out, cout), dtype=y.dtype, device=y.device) if out is None else out
    dt = _DTYPES[y.dtype]
    nbytes = int(lib().spc_conv_workspace_size(K, y.shape[0], n_out, cy, cout, dt))
    if nbytes and (ws is None or ws.numel() < nbytes):
        ws = _workspace(nbytes, y.device)
    code = lib().spc_conv_inverse(_ptr(y), _ptr(w), _ptr(b), _ptr(m), _ptr(mask_t), _ptr(perm), K,
                                  y.shape[0], n_out, cy, cout, dt, precision, _ptr(o),
                                  _ptr(status), _ptr(ws), 0 if ws is None else ws.numel(),
                                  _stream(y.device))
    _check(code, "spc_conv_inverse")
    return o


def spc_conv_fwd_int8(x: torch.Tensor, w: torch.Tensor, scale: torch.Tensor,
                      bias: Optional[torch.Tensor], imap: Optional[torch.Tensor],
                      mask: Optional[torch.Tensor] = None, perm: Optional[torch.Tensor] = None,
                      add: Optional[torch.Tensor] = None, add_scale: float = 0.0,
                      act: int = SPC_ACT_NONE, n_out: Optional[int] = None,
                      out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quantized forward: int8 x [n_in, cin], int8 w [K, cin, cout], fp32 per-channel
    scale and bias, optional int8 residual `add` with `add_scale`, optional ReLU;
    returns int8 [n_out, cout].  `perm` / `mask` from spc_map_row_order(imap)
    group rows by offset mask (spconv's do_sort); None keeps map order."""
    x = _cuda(x, "x")
    w = _cuda(w, "w")
    assert x.dtype == torch.int8 and w.dtype == torch.int8
    sc = _cuda(scale, "scale").to(torch.float32).contiguous()
    b = _cuda(bias, "bias").to(torch.float32).contiguous() if bias is not None else None
    K, cin, cout = w.shape
    if imap is not None:
        imap = _cuda(imap, "imap")
        n_out = imap.shape[1]
    elif n_out is None:
        n_out = x.shape[0]
    y = torch.empty((n_out, cout), dtype=torch.int8, device=x.device) if out is None else out
    nbytes = int(lib().spc_conv_int8_workspace_size(K, cin, cout))
    if ws is None or ws.numel() < nbytes:
        ws = _workspace(max(nbytes, 256), x.device)
    code = lib().spc_conv_fwd_int8(_ptr(x), _ptr(w), _ptr(sc), _ptr(b), _ptr(imap), _ptr(mask),
                                   _ptr(perm), K, x.shape[0], n_out, cin, cout, _ptr(add),
                                   float(add_scale), act, _ptr(y), _ptr(status), _ptr(ws),
                                   ws.numel(), _stream(x.device))
    _check(code, "spc_conv_fwd_int8")
    return y


def spc_conv_dgrad(dy: torch.Tensor, w: torch.Tensor, map_: Optional[torch.Tensor], kind: int,
                   n_in: int, precision: int = SPC_PREC_EXACT, mask: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None,
                   perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx[i] = sum over pairs imap[k, o] = i of W[k] dy[o]; `perm` orders the
    input-row tiles (for a submanifold map, the forward's row order)."""
    dy = _cuda(dy, "dy")
    w = _cuda(w, "w").to(dy.dtype)
    K, cin, cout = w.shape
    m = _cuda(map_, "map") if map_ is not None else None
    dx = torch.empty((n_in, cin), dtype=dy.dtype, device=dy.device) if out is None else out
    dt = _DTYPES[dy.dtype]
    code = lib().spc_conv_dgrad(_ptr(dy), _ptr(w), _ptr(m), kind, _ptr(mask), _ptr(perm), K, n_in,
                                dy.shape[0], cin, cout, dt, precision, _ptr(dx), _ptr(status),
                                None, 0, _stream(dy.device))
    _check(code, "spc_conv_dgrad")
    return dx


def spc_conv_wgrad(x: torch.Tensor, dy: torch.Tensor, imap: Optional[torch.Tensor], K: int,
                   precision: int = SPC_PREC_EXACT, out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dW[k] = sum over pairs of x[imap[k, o]]^T dy[o], float32 [K, cin, cout]."""
    x = _cuda(x, "x")
    dy = _cuda(dy, "dy").to(x.dtype)
    m = _cuda(imap, "imap") if imap is not None else None
    cin, cout = x.shape[1], dy.shape[1]
    dw = torch.empty((K, cin, cout), dtype=torch.float32, device=x.device) if out is None else out
    dt = _DTYPES[x.dtype]
    nbytes = int(lib().spc_conv_wgrad_workspace_size(K, x.shape[0], dy.shape[0], cin, cout, dt))
    if ws is None or ws.numel() < nbytes:
        ws = _workspace(nbytes, x.device)
    code = lib().spc_conv_wgrad(_ptr(x), _ptr(dy), _ptr(m), K, x.shape[0], dy.shape[0], cin, cout,
                                dt, precision, _ptr(dw), _ptr(status), _ptr(ws), ws.numel(),
                                _stream(x.device))
    _check(code, "spc_conv_wgrad")
    return dw


# The layers between convolutions.  Their calls can be shorter than a few microseconds on the
# device, so what does not need a tensor operation here does not get one.

def _int32(t: torch.Tensor, name: str) -> torch.Tensor:
    """Whole numbers as int32.  One that 32 bits do not hold becomes the nearest that they do, which is out of
    every range here as the number itself is (its low half might not be)."""
    if t.is_floating_point() or t.is_complex():
        raise ValueError(f"{name} must hold whole numbers, not {t.dtype}")
    if t.dtype is torch.uint32 or t.dtype is torch.uint64:
        t = t.to(torch.int64)  # from 2^63 on: below zero
    return (t.clamp(-2 ** 31, 2 ** 31 - 1) if t.dtype is torch.int64 else t).to(torch.int32)


def _typed(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    """A contiguous CUDA tensor of the given type."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        t = _int32(t, name) if dtype is torch.int32 else t.to(dtype)
    return t if t.is_contiguous() else t.contiguous()


def _values(t: torch.Tensor, name: str) -> torch.Tensor:
    """A feature tensor of a supported type."""
    t = _cuda(t, name)
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    return t


def _expect(t: torch.Tensor, shape, name: str):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _optional(t: Optional[torch.Tensor], dtype, shape, name: str):
    """(tensor, pointer) of an optional argument."""
    if t is None:
        return None, None
    t = _typed(t, dtype, name)
    _expect(t, shape, name)
    return t, t.data_ptr()


def _status(t: Optional[torch.Tensor]):
    """The pointer of a status word, which kernels write to."""
    if t is None:
        return None
    if not t.is_cuda or t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError("status must be an int32 CUDA tensor of one element")
    return t.data_ptr()


def _room(ws: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    """The caller's workspace where it is large enough, or a new one."""
    if ws is None:
        return _workspace(nbytes, device)
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor")
    return ws if ws.numel() >= nbytes else _workspace(nbytes, device)


def _result(out: Optional[torch.Tensor], shape, dtype, device, name: str) -> torch.Tensor:
    """The caller's output buffer, checked, or a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.shape != shape or out.dtype is not dtype or out.device != device or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def spc_row_segments(ids: torch.Tensor, segments: int, with_order: bool = True,
                     out: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None):
    """Rows grouped by a small key: (seg [segments + 1], order [n] or None), both int32.

    `ids` [n] is the key of each row (a column of a coordinate array is read in
    place); rows whose key lies outside [0, segments) come last in `order`.
    Pass `out` (seg), `order` and `ws` to call without allocating."""
    if ids.dim() != 1:
        raise ValueError("ids must have one dimension")
    if not ids.is_cuda:
        raise ValueError("ids must be a CUDA tensor")
    if ids.dtype is not torch.int32:
        ids = _int32(ids, "ids")
    n, dev = ids.shape[0], ids.device
    stride = ids.stride(0) if n > 1 else 1
    if stride < 1:
        ids, stride = ids.contiguous(), 1
    seg = _result(out, (segments + 1,), torch.int32, dev, "out")
    if with_order:
        order = _result(order, (n,), torch.int32, dev, "order")
    L = lib()
    nbytes = L.spc_row_segments_workspace_size(n, segments)
    ws = _room(ws, nbytes, dev)
    code = L.spc_row_segments(ids.data_ptr(), stride, n, segments, seg.data_ptr(),
                              order.data_ptr() if with_order else None, ws.data_ptr(), ws.numel(), _stream(dev))
    _check(code, "spc_row_segments")
    return seg, (order if with_order else None)


def spc_group_norm_fwd(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                       seg: torch.Tensor, groups: int, order: Optional[torch.Tensor] = None,
                       eps: float = 1e-5, act: int = SPC_ACT_NONE, out: Optional[torch.Tensor] = None,
                       mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """y = act(gamma (x - mean) rstd + beta) with statistics per segment (sample) and group of
    channels: returns (y [n, C], mean [S, groups], rstd [S, groups]).

    `seg` / `order` from spc_row_segments (order None: rows lie in grouped order);
    pass `out`, `mean`, `rstd` and `ws` to call without allocating."""
    x = _values(x, "x")
    n, c = x.shape
    dev, dt = x.device, _DTYPES[x.dtype]
    seg = _typed(seg, torch.int32, "seg")
    segments = seg.shape[0] - 1
    order, order_p = _optional(order, torch.int32, (n,), "order")
    gamma, gamma_p = _optional(gamma, torch.float32, (c,), "gamma")
    beta, beta_p = _optional(beta, torch.float32, (c,), "beta")
    y = _result(out, (n, c), x.dtype, dev, "out")
    mean = _result(mean, (segments, groups), torch.float32, dev, "mean")
    rstd = _result(rstd, (segments, groups), torch.float32, dev, "rstd")
    L = lib()
    nbytes = L.spc_group_norm_workspace_size(n, c, segments, groups, dt)
    ws = _room(ws, nbytes, dev)
    code = L.spc_group_norm_fwd(x.data_ptr(), gamma_p, beta_p, seg.data_ptr(), order_p, segments, n, c, groups,
                                eps, act, dt, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _status(status),
                                ws.data_ptr(), ws.numel(), _stream(dev))
    _check(code, "spc_group_norm_fwd")
    return y, mean, rstd


def spc_group_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor],
                       beta: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor,
                       seg: torch.Tensor, groups: int, order: Optional[torch.Tensor] = None,
                       act: int = SPC_ACT_NONE, out: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Gradients of spc_group_norm_fwd: (dx [n, C], dgamma [C] fp32, dbeta [C] fp32).
    `mean` and `rstd` come from the forward call."""
    x = _values(x, "x")
    n, c = x.shape
    dev, dt = x.device, _DTYPES[x.dtype]
    dy = _typed(dy, x.dtype, "dy")
    _expect(dy, (n, c), "dy")
    seg = _typed(seg, torch.int32, "seg")
    segments = seg.shape[0] - 1
    order, order_p = _optional(order, torch.int32, (n,), "order")
    gamma, gamma_p = _optional(gamma, torch.float32, (c,), "gamma")
    beta, beta_p = _optional(beta, torch.float32, (c,), "beta")
    mean, mean_p = _optional(mean, torch.float32, (segments, groups), "mean")
    rstd, rstd_p = _optional(rstd, torch.float32, (segments, groups), "rstd")
    dx = _result(out, (n, c), x.dtype, dev, "out")
    dgamma = torch.empty(c, dtype=torch.float32, device=dev)
    dbeta = torch.empty(c, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.spc_group_norm_workspace_size(n, c, segments, groups, dt)
    ws = _room(ws, nbytes, dev)
    code = L.spc_group_norm_bwd(dy.data_ptr(), x.data_ptr(), gamma_p, beta_p, mean_p, rstd_p, seg.data_ptr(),
                                order_p, segments, n, c, groups, act, dt, dx.data_ptr(), dgamma.data_ptr(),
                                dbeta.data_ptr(), _status(status), ws.data_ptr(), ws.numel(), _stream(dev))
    _check(code, "spc_group_norm_bwd")
    return dx, dgamma, dbeta


def _rng(rng: torch.Tensor) -> torch.Tensor:
    rng = _cuda(rng, "rng")
    if (rng.dtype is not torch.int64 and rng.dtype is not torch.uint64) or rng.numel() != 2:
        raise ValueError("rng must hold two 64-bit integers: seed and offset")
    return rng


def spc_dropout_fwd(x: torch.Tensor, p: float, rng: torch.Tensor,
                    residual: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = residual + (x / (1 - p) where kept, else 0).  `rng` [2] int64 on the device holds
    seed and offset; the mask is computed from them and the element's index, never stored."""
    x = _values(x, "x")
    residual, residual_p = _optional(residual, x.dtype, x.shape, "residual")
    rng = _rng(rng)
    y = torch.empty_like(x) if out is None else _result(out, x.shape, x.dtype, x.device, "out")
    code = lib().spc_dropout_fwd(x.data_ptr(), residual_p, x.numel(), p, rng.data_ptr(), _DTYPES[x.dtype],
                                 y.data_ptr(), _stream(x.device))
    _check(code, "spc_dropout_fwd")
    return y


def spc_dropout_bwd(dy: torch.Tensor, p: float, rng: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx = dy / (1 - p) where the forward call with this rng and p kept the element, else 0."""
    dy = _values(dy, "dy")
    rng = _rng(rng)
    dx = torch.empty_like(dy) if out is None else _result(out, dy.shape, dy.dtype, dy.device, "out")
    code = lib().spc_dropout_bwd(dy.data_ptr(), dy.numel(), p, rng.data_ptr(), _DTYPES[dy.dtype], dx.data_ptr(),
                                 _stream(dy.device))
    _check(code, "spc_dropout_bwd")
    return dx


def _positions(x_rows, y_rows, rows: int):
    """Row lists with their pointers, and the number of positions (a list's length, else the operand's rows)."""
    m = rows
    if x_rows is not None:
        m = x_rows.shape[0]
    elif y_rows is not None:
        m = y_rows.shape[0]
    x_rows, x_p = _optional(x_rows, torch.int32, (m,), "x_rows")
    y_rows, y_p = _optional(y_rows, torch.int32, (m,), "y_rows")
    return x_rows, x_p, y_rows, y_p, m


def _grouped_ws(ws, segments, m, cin, cout, dt, listed, device):
    nbytes = lib().spc_grouped_workspace_size(segments, m, cin, cout, dt, listed)
    if not nbytes and ws is None:
        return None, None, 0
    ws = _room(ws, nbytes, device)
    return ws, ws.data_ptr(), ws.numel()


def spc_grouped_fwd(x: torch.Tensor, w: torch.Tensor, seg: torch.Tensor,
                    x_rows: Optional[torch.Tensor] = None, y_rows: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[y_rows[r]] = x[x_rows[r]] W[g] for the positions r of each segment (expert) g:
    w [segments, cin, cout]; returns y [m, cout].  A list left out means row r at position r."""
    x = _values(x, "x")
    w = _typed(w, x.dtype, "w")
    segments, cin, cout = w.shape
    n_x, dev, dt = x.shape[0], x.device, _DTYPES[x.dtype]
    _expect(x, (n_x, cin), "x")
    seg = _typed(seg, torch.int32, "seg")
    _expect(seg, (segments + 1,), "seg")
    x_rows, x_p, y_rows, y_p, m = _positions(x_rows, y_rows, n_x)
    y = _result(out, (m, cout), x.dtype, dev, "out")
    ws_p, ws_n = (None, 0) if ws is None else (_room(ws, 0, dev).data_ptr(), ws.numel())  # only the gradient by w needs one
    code = lib().spc_grouped_fwd(x.data_ptr(), w.data_ptr(), seg.data_ptr(), x_p, y_p, segments, n_x, m, cin, cout,
                                 dt, y.data_ptr(), _status(status), ws_p, ws_n, _stream(dev))
    _check(code, "spc_grouped_fwd")
    return y


def spc_grouped_dgrad(dy: torch.Tensor, w: torch.Tensor, seg: torch.Tensor,
                      x_rows: Optional[torch.Tensor] = None, y_rows: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx[x_rows[r]] = dy[y_rows[r]] W[g]^T; returns dx [m, cin].  Where the forward's x_rows
    repeat rows, pass the list of slots instead and sum a row's slots."""
    dy = _values(dy, "dy")
    w = _typed(w, dy.dtype, "w")
    segments, cin, cout = w.shape
    n_y, dev, dt = dy.shape[0], dy.device, _DTYPES[dy.dtype]
    _expect(dy, (n_y, cout), "dy")
    seg = _typed(seg, torch.int32, "seg")
    _expect(seg, (segments + 1,), "seg")
    x_rows, x_p, y_rows, y_p, m = _positions(x_rows, y_rows, n_y)
    dx = _result(out, (m, cin), dy.dtype, dev, "out")
    ws_p, ws_n = (None, 0) if ws is None else (_room(ws, 0, dev).data_ptr(), ws.numel())  # only the gradient by w needs one
    code = lib().spc_grouped_dgrad(dy.data_ptr(), w.data_ptr(), seg.data_ptr(), x_p, y_p, segments, n_y, m, cin, cout,
                                   dt, dx.data_ptr(), _status(status), ws_p, ws_n, _stream(dev))
    _check(code, "spc_grouped_dgrad")
    return dx


def spc_grouped_wgrad(x: torch.Tensor, dy: torch.Tensor, seg: torch.Tensor,
                      x_rows: Optional[torch.Tensor] = None, y_rows: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dW[g] = sum over the positions r of segment g of x[x_rows[r]]^T dy[y_rows[r]],
    float32 [segments, cin, cout]."""
    x = _values(x, "x")
    dy = _typed(dy, x.dtype, "dy")
    (n_x, cin), (n_y, cout) = x.shape, dy.shape
    dev, dt = x.device, _DTYPES[x.dtype]
    seg = _typed(seg, torch.int32, "seg")
    segments = seg.shape[0] - 1
    x_rows, x_p, y_rows, y_p, m = _positions(x_rows, y_rows, max(n_x, n_y))
    dw = _result(out, (segments, cin, cout), torch.float32, dev, "out")
    ws, ws_p, ws_n = _grouped_ws(ws, segments, m, cin, cout, dt, x_p is not None or y_p is not None, dev)
    code = lib().spc_grouped_wgrad(x.data_ptr(), dy.data_ptr(), seg.data_ptr(), x_p, y_p, segments, n_x, n_y, m, cin,
                                   cout, dt, dw.data_ptr(), _status(status), ws_p, ws_n, _stream(dev))
    _check(code, "spc_grouped_wgrad")
    return dw


# A transformer block's layers.  Their tensors lie on one device, whichever is current.

def _held(sizes: int, where: str):
    """Refuses sizes and choices (or'ed together) that the library takes in 32 bits and that these do not hold, of which
    ctypes would pass the low half."""
    if not 0 <= sizes <= 0x7fffffff:
        raise SpcError(SPC_ERR_INVALID_ARG, where)


def _one_device(dev, *tensors):
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, expected {dev}")


def _launch(dev, f, *args):
    """Calls a C entry with `dev` as the current device and its current stream as the last argument."""
    if torch._C._cuda_getDevice() == dev.index:
        return f(*args, _stream(dev))
    with torch.cuda.device(dev):
        return f(*args, _stream(dev))


def _matrix(t: torch.Tensor, name: str) -> torch.Tensor:
    t = _values(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t


def _head_rows(t: torch.Tensor, name: str):
    """(tensor, elements from row to row) of rows [heads, d]; what is not laid out so is copied."""
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [rows, heads, channels]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    n, heads, d = t.shape
    ld, between, step = t.stride()
    if n > 1 and ld < heads * d or heads > 1 and between != d or d > 1 and step != 1:
        t, ld = t.contiguous(), heads * d
    return t, ld if n > 1 else heads * d


def _head_result(out: Optional[torch.Tensor], shape, dtype, device, name: str):
    """(tensor, elements from row to row) of a caller's output, checked, or of a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device), shape[1] * shape[2]
    if out.shape != shape or out.dtype is not dtype or out.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    laid, ld = _head_rows(out, name)
    if laid is not out:
        raise ValueError(f"{name}'s rows must hold their heads' channels one after the other")
    return out, ld


def spc_layer_norm_fwd(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float = 1e-5,
                       out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                       rstd: Optional[torch.Tensor] = None):
    """y = gamma (x - mean) rstd + beta with the statistics of each row of x [n, C]: returns (y, mean [n],
    rstd [n]).  Pass `out`, `mean` and `rstd` to call without allocating."""
    x = _matrix(x, "x")
    n, c = x.shape
    _held(c, "spc_layer_norm_fwd")
    dev = x.device
    gamma, gamma_p = _optional(gamma, torch.float32, (c,), "gamma")
    beta, beta_p = _optional(beta, torch.float32, (c,), "beta")
    _one_device(dev, gamma, beta)
    y = _result(out, (n, c), x.dtype, dev, "out")
    mean = _result(mean, (n,), torch.float32, dev, "mean")
    rstd = _result(rstd, (n,), torch.float32, dev, "rstd")
    code = _launch(dev, lib().spc_layer_norm_fwd, x.data_ptr(), gamma_p, beta_p, n, c, eps, _DTYPES[x.dtype], y.data_ptr(),
                   mean.data_ptr(), rstd.data_ptr())
    _check(code, "spc_layer_norm_fwd")
    return y, mean, rstd


def spc_layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor,
                       rstd: torch.Tensor, out: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                       dbeta: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Gradients of spc_layer_norm_fwd: (dx [n, C], dgamma [C] fp32, dbeta [C] fp32).  `mean` and `rstd` come from
    the forward call."""
    x = _matrix(x, "x")
    n, c = x.shape
    _held(c, "spc_layer_norm_bwd")
    dev = x.device
    dy = _typed(dy, x.dtype, "dy")
    _expect(dy, (n, c), "dy")
    gamma, gamma_p = _optional(gamma, torch.float32, (c,), "gamma")
    mean, mean_p = _optional(mean, torch.float32, (n,), "mean")
    rstd, rstd_p = _optional(rstd, torch.float32, (n,), "rstd")
    _one_device(dev, dy, gamma, mean, rstd, ws)
    dx = _result(out, (n, c), x.dtype, dev, "out")
    dgamma = _result(dgamma, (c,), torch.float32, dev, "dgamma")
    dbeta = _result(dbeta, (c,), torch.float32, dev, "dbeta")
    L = lib()
    ws = _room(ws, _launch_size(dev, L.spc_layer_norm_workspace_size, n, c), dev)
    code = _launch(dev, L.spc_layer_norm_bwd, dy.data_ptr(), x.data_ptr(), gamma_p, mean_p, rstd_p, n, c, _DTYPES[x.dtype],
                   dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), ws.numel())
    _check(code, "spc_layer_norm_bwd")
    return dx, dgamma, dbeta


def _launch_size(dev, f, *args) -> int:
    """A workspace's size, which may depend on the device."""
    if torch._C._cuda_getDevice() == dev.index:
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


@functools.lru_cache(maxsize=64, typed=True)
def _three(*pairs):
    """(C array, sum) of the numbers of turned pairs of channels for z, y and x."""
    try:
        t = tuple(operator.index(p) for p in pairs)
    except TypeError:
        t = ()
    if len(t) != 3 or min(t) < 0 or max(t) > 0x7fffffff:
        raise ValueError("pairs must hold the number of turned pairs of channels for z, y and x, whole and not negative")
    return _I3(*t), sum(t)


def spc_rope_steps(pairs: Sequence[int], base: float = 10000.0) -> torch.Tensor:
    """Steps of spc_rope_fwd for base^(-j / pairs[axis]) radians a cell, j = 0 .. pairs[axis] - 1: a CPU tensor
    [sum(pairs)] int64, 2^64 to a full turn.  Computed once, kept by the caller."""
    counts, turned = _three(*pairs)
    steps = torch.empty(turned, dtype=torch.int64)
    _check(lib().spc_rope_steps(counts, base, steps.data_ptr() if turned else None), "spc_rope_steps")
    return steps


def _rope(f, name: str, x: torch.Tensor, coords: torch.Tensor, steps: torch.Tensor, pairs, out):
    x, ldx = _head_rows(x, "x")
    n, heads, d = x.shape
    _held(heads | d, name)
    dev = x.device
    counts, turned = _three(*pairs)
    if not coords.is_cuda or coords.dtype is not torch.int32:
        raise ValueError("coords must be an int32 CUDA tensor")
    _expect(coords, (n, 4), "coords")
    coords = coords if coords.is_contiguous() else coords.contiguous()
    if steps.is_cuda or steps.dtype is not torch.int64 or not steps.is_contiguous():
        raise ValueError("steps must be a contiguous int64 CPU tensor (spc_rope_steps)")
    _expect(steps, (turned,), "steps")
    _one_device(dev, coords)
    y, ldy = _head_result(out, (n, heads, d), x.dtype, dev, "out")
    code = _launch(dev, f, x.data_ptr(), ldx, coords.data_ptr(), counts, steps.data_ptr() if turned else None, n, heads, d,
                   _DTYPES[x.dtype], y.data_ptr(), ldy)
    _check(code, name)
    return y


def spc_rope_fwd(x: torch.Tensor, coords: torch.Tensor, steps: torch.Tensor, pairs: Sequence[int],
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions: pairs (2i, 2i + 1) of the channels of each head of x [n, heads, d] turned by the voxel's
    cell times the pair's step, the first pairs[0] pairs by z, the next pairs[1] by y, the next pairs[2] by x of
    coords [n, 4] int32 (b, z, y, x); the rest is copied.  A slice of a projection's rows (qkv[:, :2 * heads]) is
    read in place; `out` may be such a slice, or x itself."""
    return _rope(lib().spc_rope_fwd, "spc_rope_fwd", x, coords, steps, pairs, out)


def spc_rope_bwd(dy: torch.Tensor, coords: torch.Tensor, steps: torch.Tensor, pairs: Sequence[int],
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of spc_rope_fwd: the same turns backwards."""
    return _rope(lib().spc_rope_bwd, "spc_rope_bwd", dy, coords, steps, pairs, out)


def spc_route_fwd(logits: torch.Tensor, top_k: int, score: int = SPC_SCORE_SOFTMAX, bias: Optional[torch.Tensor] = None,
                  groups: int = 1, top_groups: int = 1, renorm: bool = True, scale: float = 1.0,
                  expert: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None):
    """The top_k experts of each token and their weights: (expert [n, top_k] int32, gate [n, top_k] fp32), best first.
    logits [n, experts]; `bias` [experts] counts in the choice only; of `groups` groups of neighbouring experts the
    top_groups best are kept (by the sum of their two best); `renorm` divides the weights by their sum.  A slot
    for which no expert is available (logits of -inf or NaN) holds -1 and weight 0."""
    logits = _matrix(logits, "logits")
    n, experts = logits.shape
    _held(experts | top_k | score | groups | top_groups, "spc_route_fwd")
    dev = logits.device
    bias, bias_p = _optional(bias, torch.float32, (experts,), "bias")
    _one_device(dev, bias)
    expert = _result(expert, (n, top_k), torch.int32, dev, "expert")
    gate = _result(gate, (n, top_k), torch.float32, dev, "gate")
    code = _launch(dev, lib().spc_route_fwd, logits.data_ptr(), bias_p, n, experts, top_k, score, groups, top_groups, bool(renorm),
                   scale, _DTYPES[logits.dtype], expert.data_ptr(), gate.data_ptr())
    _check(code, "spc_route_fwd")
    return expert, gate


def spc_route_bwd(dgate: torch.Tensor, logits: torch.Tensor, expert: torch.Tensor, score: int = SPC_SCORE_SOFTMAX,
                  renorm: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of spc_route_fwd's weights by the logits, [n, experts] of their type, for the experts that the
    forward call chose."""
    logits = _matrix(logits, "logits")
    n, experts = logits.shape
    dev = logits.device
    expert = _typed(expert, torch.int32, "expert")
    if expert.dim() != 2:
        raise ValueError("expert must have shape [n, top_k]")
    top_k = expert.shape[1]
    _held(experts | top_k | score, "spc_route_bwd")
    _expect(expert, (n, top_k), "expert")
    dgate = _typed(dgate, torch.float32, "dgate")
    _expect(dgate, (n, top_k), "dgate")
    _one_device(dev, expert, dgate, status)
    dlogits = _result(out, (n, experts), logits.dtype, dev, "out")
    code = _launch(dev, lib().spc_route_bwd, dgate.data_ptr(), logits.data_ptr(), expert.data_ptr(), n, experts, top_k, score,
                   bool(renorm), scale, _DTYPES[logits.dtype], dlogits.data_ptr(), _status(status))
    _check(code, "spc_route_bwd")
    return dlogits


def _attention_args(q, k, v, seg, seg_k, scale):
    q, ldq = _head_rows(q, "q")
    (nq, hq, d), dev = q.shape, q.device
    k, ldk = _head_rows(k if k.dtype is q.dtype else k.to(q.dtype), "k")
    nk, hk = k.shape[:2]
    _expect(k, (nk, hk, d), "k")
    v, ldv = _head_rows(v if v.dtype is q.dtype else v.to(q.dtype), "v")
    _expect(v, (nk, hk, d), "v")
    seg = _typed(seg, torch.int32, "seg")
    if seg.dim() != 1 or seg.shape[0] < 2:
        raise ValueError("seg must hold segments + 1 offsets")
    if seg_k is None:
        if nk != nq:
            raise ValueError("without seg_k there are as many keys as queries")
        seg_k = seg
    else:
        seg_k = _typed(seg_k, torch.int32, "seg_k")
        _expect(seg_k, seg.shape, "seg_k")
    _one_device(dev, k, v, seg, seg_k)
    segments = seg.shape[0] - 1
    _held(hq | hk | d | segments, "spc_attention")
    return q, ldq, k, ldk, v, ldv, seg, seg_k, segments, nq, nk, hq, hk, d, max(d, 1) ** -0.5 if scale is None else scale, dev


def spc_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seg: torch.Tensor,
                      seg_k: Optional[torch.Tensor] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None):
    """Attention of each query to the keys of its own segment: (o [nq, hq, d], lse [nq, hq] fp32).

    q [nq, hq, d]; k, v [nk, hk, d], hk dividing hq (query head h reads key head h // (hq // hk)); slices of a
    projection's rows are read in place.  `seg` [segments + 1] int32 holds the offsets of the queries'
    segments, `seg_k` those of the keys (None: the same rows).  scale None: d^-0.5.  A query without keys
    gives 0 and lse -inf.  Pass `out`, `lse` and `ws` to call without allocating."""
    q, ldq, k, ldk, v, ldv, seg, seg_k, segments, nq, nk, hq, hk, d, scale, dev = _attention_args(q, k, v, seg, seg_k, scale)
    _one_device(dev, ws, status)
    o, ldo = _head_result(out, (nq, hq, d), q.dtype, dev, "out")
    lse = _result(lse, (nq, hq), torch.float32, dev, "lse")
    L, dt = lib(), _DTYPES[q.dtype]
    nbytes = _launch_size(dev, L.spc_attention_workspace_size, nq, nk, segments, hq, hk, d, dt, 0)
    if nbytes or ws is not None:
        ws = _room(ws, nbytes, dev)
    code = _launch(dev, L.spc_attention_fwd, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, seg.data_ptr(),
                   seg_k.data_ptr(), segments, nq, nk, hq, hk, d, scale, dt, o.data_ptr(), ldo, lse.data_ptr(),
                   _status(status), _ptr(ws), 0 if ws is None else ws.numel())
    _check(code, "spc_attention_fwd")
    return o, lse


def spc_attention_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                      lse: torch.Tensor, seg: torch.Tensor, seg_k: Optional[torch.Tensor] = None,
                      scale: Optional[float] = None, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                      dv: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None):
    """Gradients of spc_attention_fwd: (dq [nq, hq, d], dk, dv [nk, hk, d]).  `o` and `lse` come from the forward
    call.  `dq`, `dk` and `dv` may be slices of one gradient of the projection's rows."""
    q, ldq, k, ldk, v, ldv, seg, seg_k, segments, nq, nk, hq, hk, d, scale, dev = _attention_args(q, k, v, seg, seg_k, scale)
    dout, lddo = _head_rows(dout if dout.dtype is q.dtype else dout.to(q.dtype), "dout")
    _expect(dout, (nq, hq, d), "dout")
    o, ldo = _head_rows(o if o.dtype is q.dtype else o.to(q.dtype), "o")
    _expect(o, (nq, hq, d), "o")
    lse, lse_p = _optional(lse, torch.float32, (nq, hq), "lse")
    _one_device(dev, dout, o, lse, ws, status)
    dq, lddq = _head_result(dq, (nq, hq, d), q.dtype, dev, "dq")
    dk, lddk = _head_result(dk, (nk, hk, d), q.dtype, dev, "dk")
    dv, lddv = _head_result(dv, (nk, hk, d), q.dtype, dev, "dv")
    L, dt = lib(), _DTYPES[q.dtype]
    ws = _room(ws, _launch_size(dev, L.spc_attention_workspace_size, nq, nk, segments, hq, hk, d, dt, 1), dev)
    code = _launch(dev, L.spc_attention_bwd, dout.data_ptr(), lddo, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
                   o.data_ptr(), ldo, lse_p, seg.data_ptr(), seg_k.data_ptr(), segments, nq, nk, hq, hk, d, scale, dt,
                   dq.data_ptr(), lddq, dk.data_ptr(), lddk, dv.data_ptr(), lddv, _status(status), ws.data_ptr(), ws.numel())
    _check(code, "spc_attention_bwd")
    return dq, dk, dv
