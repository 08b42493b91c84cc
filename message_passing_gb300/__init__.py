"""Python binding of libe3gb.so (include/e3gb.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; PyTorch provides device
memory and streams. The functions keep the C names without the ``e3gb_`` prefix and take
torch tensors. If the library is missing or fails to load, importing the functions raises
(there is no CPU path).

Operations follow "e3j: An efficient and open-source backend for Euclidean equivariant
operations on GPU and TPU", App. E.1 Eq. (10)-(16); see include/e3gb.h for layouts.
"""
from __future__ import annotations

import array
import ctypes
import os
from dataclasses import dataclass, field
from functools import lru_cache
from operator import attrgetter

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libe3gb.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_BAD_GRAPH, ERR_DEVICE_INDEX = range(6)
F32, BF16 = 0, 1
PATHS_SUMMED, PATHS_SEPARATE = 0, 1

# every symbol include/e3gb.h declares
SYMBOLS = (
    "e3gb_table_create", "e3gb_table_destroy", "e3gb_table_info", "e3gb_table_paths",
    "e3gb_table_coefficients", "e3gb_config_count", "e3gb_config_describe", "e3gb_sh_forward",
    "e3gb_sh_backward",
    "e3gb_tp_forward", "e3gb_tp_backward", "e3gb_graph_prepare_workspace_bytes",
    "e3gb_graph_prepare", "e3gb_graph_prepare_static", "e3gb_conv_forward", "e3gb_conv_backward",
    "e3gb_conv_double_backward", "e3gb_coo_tp_forward", "e3gb_coo_tp_backward",
    "e3gb_radial_hidden", "e3gb_radial_backward", "e3gb_conv_forward_radial", "e3gb_conv_backward_radial",
    "e3gb_conv_forward_split_workspace_bytes", "e3gb_conv_forward_split",
    "e3gb_layer_norm_forward", "e3gb_layer_norm_backward_workspace_bytes", "e3gb_layer_norm_backward",
    "e3gb_irreps_norm_forward", "e3gb_irreps_norm_backward_workspace_bytes", "e3gb_irreps_norm_backward",
    "e3gb_adamw_create", "e3gb_adamw_destroy", "e3gb_adamw_info", "e3gb_adamw_plan", "e3gb_adamw_step",
    "e3gb_check_device_status", "e3gb_last_error", "e3gb_version",
)

# hidden width the radial convolution kernels are built for
RADIAL_HIDDEN = 8


class E3GBError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"e3gb status {status}: {msg}")
        self.status = status


class _Irreps(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("l", ctypes.POINTER(ctypes.c_int32)),
                ("parity", ctypes.POINTER(ctypes.c_int32)), ("mul", ctypes.c_int32)]


class _AdamwRates(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("max_norm", ctypes.c_double), ("step", ctypes.c_int64),
                ("seed", ctypes.c_uint32)]


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libe3gb.so (built by message_passing_gb300.build). Raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with message_passing_gb300.build.build()")
    lib = ctypes.CDLL(p)
    i32, i64, vp, f32, szt = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    P32 = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "e3gb_table_create": (i32, [ctypes.POINTER(_Irreps), i32, i32, i32, ctypes.POINTER(vp)]),
        "e3gb_table_destroy": (i32, [vp]),
        "e3gb_table_info": (i32, [vp, P32, P32, P32, P32, P32, P32]),
        "e3gb_table_paths": (i32, [vp, P32]),
        "e3gb_table_coefficients": (i32, [vp, ctypes.POINTER(ctypes.c_double)]),
        "e3gb_config_count": (i32, []),
        "e3gb_config_describe": (i32, [i32, P32, P32, P32, P32, P32, P32]),
        "e3gb_sh_forward": (i32, [i32, i64, vp, vp, i32, vp]),
        "e3gb_sh_backward": (i32, [i32, i64, vp, vp, vp, i32, vp]),
        "e3gb_tp_forward": (i32, [vp, i64, vp, vp, vp, vp, i32, vp]),
        "e3gb_tp_backward": (i32, [vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp]),
        "e3gb_graph_prepare_workspace_bytes": (szt, [i64, i64]),
        "e3gb_graph_prepare": (i32, [i64, i64, vp, vp, vp, vp, vp, vp, szt, vp]),
        "e3gb_graph_prepare_static": (i32, [i64, i64, vp, vp, vp, vp, vp, vp]),
        "e3gb_conv_forward": (i32, [vp, i64, i64, vp, vp, vp, vp, vp, f32, i64, vp, i32, vp]),
        "e3gb_conv_backward": (i32, [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, f32, i64, vp, vp, vp, i32, vp]),
        "e3gb_conv_double_backward": (i32, [vp, i64, i64] + [vp] * 5 + [vp] * 7 + [f32, i64] + [vp] * 4
                                      + [i32, vp]),
        "e3gb_coo_tp_forward": (i32, [i64, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp]),
        "e3gb_coo_tp_backward": (i32, [i64, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                       vp]),
        "e3gb_radial_hidden": (i32, [i64, vp, vp, i32, i32, f32, vp, vp]),
        "e3gb_radial_backward": (i32, [i64, vp, vp, i32, i32, f32, vp, vp, i32, vp]),
        "e3gb_conv_forward_radial": (i32, [vp, i64, i64, vp, vp, vp, vp, vp, vp, i32, f32, i64, vp, i32, vp]),
        "e3gb_conv_backward_radial": (i32, [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp, f32, i64, vp, vp, vp,
                                            i32, vp]),
        "e3gb_conv_forward_split_workspace_bytes": (szt, [vp, i64, i64, i32]),
        "e3gb_conv_forward_split": (i32, [vp, i64, i64, vp, vp, vp, vp, vp, f32, i64, i32, vp, vp, szt, i32, vp]),
        "e3gb_layer_norm_forward": (i32, [i64, i64, vp, i64, i32, vp, vp, f32, vp, i64, i32, vp, vp]),
        "e3gb_layer_norm_backward_workspace_bytes": (szt, [i64, i64]),
        "e3gb_layer_norm_backward": (i32, [i64, i64, vp, i64, i32, vp, vp, vp, i64, i32, vp, i64, i32, vp, vp, vp, szt,
                                           vp]),
        "e3gb_irreps_norm_forward": (i32, [vp, i64, vp, i32, vp, vp, f32, vp, i32, vp, vp]),
        "e3gb_irreps_norm_backward_workspace_bytes": (szt, [vp, i64]),
        "e3gb_irreps_norm_backward": (i32, [vp, i64, vp, i32, vp, vp, vp, i32, vp, i32, vp, vp, vp, szt, vp]),
        "e3gb_adamw_create": (i32, [i32, vp, vp, vp, vp, i32, ctypes.POINTER(vp)]),
        "e3gb_adamw_destroy": (i32, [vp]),
        "e3gb_adamw_info": (i32, [vp, ctypes.POINTER(i64), ctypes.POINTER(szt), ctypes.POINTER(szt), vp]),
        "e3gb_adamw_plan": (i32, [vp, vp]),
        "e3gb_adamw_step": (i32, [vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, szt, vp]),
        "e3gb_check_device_status": (i32, [vp, P32]),
        "e3gb_last_error": (ctypes.c_char_p, []),
        "e3gb_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != OK:
        raise E3GBError(status, load().e3gb_last_error().decode())


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(*ts):
    import torch
    dt = {t.dtype for t in ts if t is not None}
    if dt == {torch.float32}:
        return F32
    if dt == {torch.bfloat16}:
        return BF16
    raise TypeError(f"tensors must all be float32 or all bfloat16, got {dt}")


def _f32_out(*ts):
    import torch
    for t in ts:
        if t is not None and t.dtype != torch.float32:
            raise TypeError("outputs are float32 in both the fp32 and the bf16 variant")


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _shape(name, t, *shape):
    """The kernels index every buffer from the table's sizes and the row/node/edge counts, so a
    buffer of another shape would be read or written out of bounds: refuse it here."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _index_len(name, t, n):
    """An index array of at least n entries (the graph index arrays hold max(E, 1))."""
    if t is not None and (t.dim() != 1 or t.shape[0] < n):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({n},) or longer")


def version() -> str:
    return load().e3gb_version().decode()


def configs() -> list[dict]:
    """The irreps configurations compiled into the library."""
    lib = load()
    out = []
    for i in range(lib.e3gb_config_count()):
        n = ctypes.c_int32()
        l = (ctypes.c_int32 * 8)()
        p = (ctypes.c_int32 * 8)()
        a, b, f = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib.e3gb_config_describe(i, ctypes.byref(n), l, p, ctypes.byref(a), ctypes.byref(b), ctypes.byref(f)))
        out.append({"blocks": [(l[k], p[k]) for k in range(n.value)], "sh_lmax": a.value,
                    "out_lmax": b.value, "per_path": bool(f.value)})
    return out


@dataclass
class Table:
    """Path table handle (e3gb_table). blocks: [(l, parity)] of x; mul: channels."""
    handle: ctypes.c_void_p
    blocks: list
    mul: int
    sh_lmax: int
    out_lmax: int
    per_path: bool
    d1: int = 0
    d2: int = 0
    n_paths: int = 0
    D: int = 0
    nnz: int = 0

    @classmethod
    def create(cls, blocks, mul: int, sh_lmax: int, out_lmax: int, per_path: bool = False) -> "Table":
        lib = load()
        n = len(blocks)
        L = (ctypes.c_int32 * max(1, n))(*[b[0] for b in blocks])
        P = (ctypes.c_int32 * max(1, n))(*[b[1] for b in blocks])
        ir = _Irreps(n, L, P, mul)
        h = ctypes.c_void_p()
        _check(lib.e3gb_table_create(ctypes.byref(ir), sh_lmax, out_lmax,
                                     PATHS_SEPARATE if per_path else PATHS_SUMMED, ctypes.byref(h)))
        t = cls(h, list(blocks), mul, sh_lmax, out_lmax, per_path)
        v = [ctypes.c_int32() for _ in range(6)]
        _check(lib.e3gb_table_info(h, *[ctypes.byref(x) for x in v]))
        t.d1, t.d2, t.n_paths, t.D, t.nnz, _ = (x.value for x in v)
        return t

    def paths(self) -> list[tuple]:
        buf = (ctypes.c_int32 * (8 * self.n_paths))()
        _check(load().e3gb_table_paths(self.handle, buf))
        return [tuple(buf[8 * i:8 * i + 8]) for i in range(self.n_paths)]

    def coefficients(self):
        import numpy as np
        buf = (ctypes.c_double * (5 * self.nnz))()
        _check(load().e3gb_table_coefficients(self.handle, buf))
        return np.frombuffer(buf, dtype=np.float64).reshape(self.nnz, 5).copy()

    def coo_records(self):
        """The table's CG tensor product as records for coo_tp_forward: (int32 [n,4] rows
        (i0, i1, i2, path), float32 [n] coefficients), host arrays."""
        import numpy as np
        xoff = np.concatenate([[0], np.cumsum([2 * l + 1 for l, _ in self.blocks])])
        paths = np.array(self.paths(), dtype=np.int64).reshape(-1, 8)
        co = self.coefficients()
        p = co[:, 0].astype(np.int64)
        rec = np.stack([paths[p, 7] + co[:, 3].astype(np.int64),            # output offset + m3
                        xoff[paths[p, 0]] + co[:, 1].astype(np.int64),      # x block offset + m1
                        paths[p, 3] ** 2 + co[:, 2].astype(np.int64),       # l2^2 + m2
                        p], axis=1).astype(np.int32)
        return np.ascontiguousarray(rec), co[:, 4].astype(np.float32)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.e3gb_table_destroy(h)
            self.handle = None


def _rows_operands(t: "Table", R: int, x, y, w, names=("x", "y", "w")):
    _shape(names[0], x, R, t.d1, t.mul)
    _shape(names[1], y, R, t.d2)
    _shape(names[2], w, R, t.n_paths, t.mul)


def _conv_operands(t: "Table", N: int, E: int, x, y, w, names=("x", "y", "w")):
    _shape(names[0], x, N, t.d1, t.mul)
    _shape(names[1], y, E, t.d2)
    _shape(names[2], w, E, t.n_paths, t.mul)


def _csc_shapes(csc, N: int, E: int):
    cp, ce, cr = csc
    _shape("csc_ptr", cp, N + 1)
    _index_len("csc_edge", ce, E)
    _index_len("csc_recv", cr, E)


def sh_forward(vec, lmax: int, out=None, dtype=None, stream=None):
    """y[n, (lmax+1)^2] = real SH of vec[n, 3] (fp32 device tensor)."""
    import torch
    _contig(vec)
    if vec.dtype != torch.float32:
        raise TypeError("vec must be float32")
    dt = dtype or torch.float32
    _shape("vec", vec, vec.shape[0], 3)
    y = out if out is not None else torch.empty((vec.shape[0], (lmax + 1) ** 2), dtype=dt, device=vec.device)
    _shape("y", y, vec.shape[0], (lmax + 1) ** 2)
    _check(load().e3gb_sh_forward(lmax, vec.shape[0], _ptr(vec), _ptr(y), _dtype(y), _stream(stream)))
    return y


def sh_backward(vec, dy, lmax: int, out=None, stream=None):
    """dvec[n, 3] (fp32) = VJP of sh_forward for the cotangent dy[n, (lmax+1)^2]."""
    import torch
    _contig(vec, dy)
    if vec.dtype != torch.float32:
        raise TypeError("vec must be float32")
    n = vec.shape[0]
    _shape("vec", vec, n, 3)
    _shape("dy", dy, n, (lmax + 1) ** 2)
    dvec = out if out is not None else torch.empty((n, 3), dtype=torch.float32, device=vec.device)
    _shape("dvec", dvec, n, 3)
    _f32_out(dvec)
    _check(load().e3gb_sh_backward(lmax, vec.shape[0], _ptr(vec), _ptr(dy), _ptr(dvec), _dtype(dy), _stream(stream)))
    return dvec


def tp_forward(t: Table, x, y, w, out=None, stream=None):
    """z[R, D, mul] (fp32) = sum over paths of w * CG(x, y) per row: x [R, d1, mul],
    y [R, d2], w [R, n_paths, mul]."""
    import torch
    _contig(x, y, w, out)
    R = x.shape[0]
    _rows_operands(t, R, x, y, w)
    z = out if out is not None else torch.empty((R, t.D, t.mul), dtype=torch.float32, device=x.device)
    _shape("z", z, R, t.D, t.mul)
    _f32_out(z)
    _check(load().e3gb_tp_forward(t.handle, x.shape[0], _ptr(x), _ptr(y), _ptr(w), _ptr(z),
                                  _dtype(x, y, w), _stream(stream)))
    return z


def tp_backward(t: Table, x, y, w, dz, out=None, stream=None):
    """(dx, dy, dw) of tp_forward for the cotangent dz [R, D, mul], all fp32, shaped like
    x, y, w."""
    import torch
    _contig(x, y, w, dz)
    R = x.shape[0]
    _rows_operands(t, R, x, y, w)
    _shape("dz", dz, R, t.D, t.mul)
    if out is None:
        f = dict(dtype=torch.float32)
        out = (torch.empty_like(x, **f), torch.empty_like(y, **f), torch.empty_like(w, **f))
    dx, dy, dw = out
    _rows_operands(t, R, dx, dy, dw, ("dx", "dy", "dw"))
    _f32_out(dx, dy, dw)
    _check(load().e3gb_tp_backward(t.handle, x.shape[0], _ptr(x), _ptr(y), _ptr(w), _ptr(dz), _ptr(dx),
                                   _ptr(dy), _ptr(dw), _dtype(x, y, w, dz), _stream(stream)))
    return dx, dy, dw


def graph_prepare_workspace_bytes(n_nodes: int, n_edges: int) -> int:
    return int(load().e3gb_graph_prepare_workspace_bytes(n_nodes, n_edges))


def graph_prepare(rowptr, sender, n_nodes: int, out=None, workspace=None, stream=None):
    """(csc_ptr, csc_edge, csc_recv) int32 device tensors."""
    import torch
    _contig(rowptr, sender)
    E = sender.shape[0]
    dev = rowptr.device
    _shape("rowptr", rowptr, n_nodes + 1)
    if out is None:
        out = (torch.empty(n_nodes + 1, dtype=torch.int32, device=dev),
               torch.empty(max(E, 1), dtype=torch.int32, device=dev),
               torch.empty(max(E, 1), dtype=torch.int32, device=dev))
    _csc_shapes(out, n_nodes, E)
    nb = graph_prepare_workspace_bytes(n_nodes, E)
    ws = workspace if workspace is not None else torch.empty(nb, dtype=torch.uint8, device=dev)
    cp, ce, cr = out
    _check(load().e3gb_graph_prepare(n_nodes, E, _ptr(rowptr), _ptr(sender) if E else None, _ptr(cp),
                                     _ptr(ce) if E else None, _ptr(cr) if E else None, _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)))
    return cp, ce, cr


STATIC_PREPARE_SCRATCH_BYTES = 4 << 20


def graph_prepare_static(rowptr, sender, n_nodes: int, out=None, stream=None):
    """graph_prepare without a workspace, for callers that cannot allocate device memory:
    the library keeps the sort's digit counts in its own static device array of
    STATIC_PREPARE_SCRATCH_BYTES (calls overlapping on the GPU race on it). Pass ``out``
    to avoid allocating the outputs here too."""
    import torch
    _contig(rowptr, sender)
    E = sender.shape[0]
    dev = rowptr.device
    _shape("rowptr", rowptr, n_nodes + 1)
    if out is None:
        out = (torch.empty(n_nodes + 1, dtype=torch.int32, device=dev),
               torch.empty(max(E, 1), dtype=torch.int32, device=dev),
               torch.empty(max(E, 1), dtype=torch.int32, device=dev))
    _csc_shapes(out, n_nodes, E)
    cp, ce, cr = out
    _check(load().e3gb_graph_prepare_static(n_nodes, E, _ptr(rowptr), _ptr(sender) if E else None, _ptr(cp),
                                            _ptr(ce) if E else None, _ptr(cr) if E else None, _stream(stream)))
    return cp, ce, cr


def conv_forward(t: Table, rowptr, sender, x, y, w, scale: float, out=None, stream=None, pad_node: int = -1):
    """m = scale * sum over each receiver's CSR edges of TP(x[sender], y, w); edges touching
    pad_node (>= 0) are padding and skipped."""
    import torch
    _contig(rowptr, sender, x, y, w)
    N, E = x.shape[0], sender.shape[0]
    _shape("rowptr", rowptr, N + 1)
    _conv_operands(t, N, E, x, y, w)
    m = out if out is not None else torch.empty((N, t.D, t.mul), dtype=torch.float32, device=x.device)
    _shape("m", m, N, t.D, t.mul)
    _f32_out(m)
    _check(load().e3gb_conv_forward(t.handle, N, E, _ptr(rowptr), _ptr(sender) if E else None, _ptr(x),
                                    _ptr(y) if E else None, _ptr(w) if E else None, float(scale), int(pad_node), _ptr(m),
                                    _dtype(x, *((y, w) if E else ())), _stream(stream)))
    return m


def conv_forward_split(t: Table, rowptr, sender, x, y, w, scale: float, chunk: int = 256, out=None, workspace=None,
                       stream=None, pad_node: int = -1):
    """conv_forward with receivers of more than `chunk` edges cut into pieces summed by separate
    warps and added in piece order (deterministic); for graphs with heavy receivers."""
    import torch
    _contig(rowptr, sender, x, y, w)
    N, E = x.shape[0], sender.shape[0]
    _shape("rowptr", rowptr, N + 1)
    _conv_operands(t, N, E, x, y, w)
    m = out if out is not None else torch.empty((N, t.D, t.mul), dtype=torch.float32, device=x.device)
    _shape("m", m, N, t.D, t.mul)
    _f32_out(m)
    nb = int(load().e3gb_conv_forward_split_workspace_bytes(t.handle, N, E, int(chunk)))
    ws = workspace if workspace is not None else torch.empty(max(nb, 16), dtype=torch.uint8, device=x.device)
    _check(load().e3gb_conv_forward_split(t.handle, N, E, _ptr(rowptr), _ptr(sender) if E else None, _ptr(x),
                                          _ptr(y) if E else None, _ptr(w) if E else None, float(scale), int(pad_node),
                                          int(chunk), _ptr(m), _ptr(ws), ws.numel() * ws.element_size(),
                                          _dtype(x, *((y, w) if E else ())), _stream(stream)))
    return m


def conv_backward(t: Table, csc, x, y, w, dm, scale: float, out=None, stream=None, pad_node: int = -1):
    """csc = graph_prepare(...) output. Returns (dx, dy, dw); padding edges (touching
    pad_node >= 0) get zero dy and dw rows."""
    import torch
    cp, ce, cr = csc
    _contig(x, y, w, dm)
    N, E = x.shape[0], y.shape[0]
    _csc_shapes(csc, N, E)
    _conv_operands(t, N, E, x, y, w)
    _shape("dm", dm, N, t.D, t.mul)
    if out is None:
        f = dict(dtype=torch.float32)
        out = (torch.empty_like(x, **f), torch.empty_like(y, **f), torch.empty_like(w, **f))
    dx, dy, dw = out
    _conv_operands(t, N, E, dx, dy, dw, ("dx", "dy", "dw"))
    _f32_out(dx, dy, dw)
    _check(load().e3gb_conv_backward(t.handle, N, E, _ptr(cp), _ptr(ce) if E else None, _ptr(cr) if E else None,
                                     _ptr(x), _ptr(y) if E else None, _ptr(w) if E else None, _ptr(dm),
                                     float(scale), int(pad_node), _ptr(dx), _ptr(dy) if E else None,
                                     _ptr(dw) if E else None,
                                     _dtype(x, dm, *((y, w) if E else ())), _stream(stream)))
    return dx, dy, dw


def radial_hidden(vec, W1, r_cut: float, out=None, stream=None):
    """h [E, hidden] = silu(bessel_basis(|vec|) @ W1): the hidden layer of the radial network
    (W1 [n_basis, hidden], fp32 device tensors)."""
    import torch
    _contig(vec, W1)
    E = vec.shape[0]
    _shape("vec", vec, E, 3)
    nb, H = W1.shape
    h = out if out is not None else torch.empty((E, H), dtype=torch.float32, device=vec.device)
    _shape("h", h, E, H)
    for n, a in (("vec", vec), ("W1", W1), ("h", h)):
        if a.dtype != torch.float32:
            raise TypeError(f"{n} must be float32")
    _check(load().e3gb_radial_hidden(E, _ptr(vec) if E else None, _ptr(W1), nb, H, float(r_cut),
                                     _ptr(h) if E else None, _stream(stream)))
    return h


def radial_backward(vec, W1, r_cut: float, dh, out=None, accumulate: bool = False, stream=None):
    """dvec [E, 3] = d<dh, h>/dvec (forces through the radial weights); accumulate adds to out."""
    import torch
    _contig(vec, W1, dh)
    E = vec.shape[0]
    nb, H = W1.shape
    _shape("vec", vec, E, 3)
    _shape("dh", dh, E, H)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((E, 3), dtype=torch.float32, device=vec.device)
    _shape("dvec", out, E, 3)
    _check(load().e3gb_radial_backward(E, _ptr(vec) if E else None, _ptr(W1), nb, H, float(r_cut),
                                       _ptr(dh) if E else None, _ptr(out) if E else None, int(bool(accumulate)),
                                       _stream(stream)))
    return out


def _radial_operands(t: "Table", E: int, h, W2):
    _shape("h", h, E, RADIAL_HIDDEN)
    _shape("W2", W2, RADIAL_HIDDEN, t.n_paths, t.mul)


def conv_forward_radial(t: Table, rowptr, sender, x, y, h, W2, scale: float, out=None, stream=None,
                        pad_node: int = -1):
    """conv_forward with w[e] = h[e] @ W2 formed inside the kernel (never stored); fp32."""
    import torch
    _contig(rowptr, sender, x, y, h, W2)
    N, E = x.shape[0], sender.shape[0]
    _shape("rowptr", rowptr, N + 1)
    _shape("x", x, N, t.d1, t.mul)
    _shape("y", y, E, t.d2)
    _radial_operands(t, E, h, W2)
    m = out if out is not None else torch.empty((N, t.D, t.mul), dtype=torch.float32, device=x.device)
    _shape("m", m, N, t.D, t.mul)
    _f32_out(m, h, W2)
    _check(load().e3gb_conv_forward_radial(t.handle, N, E, _ptr(rowptr), _ptr(sender) if E else None, _ptr(x),
                                           _ptr(y) if E else None, _ptr(h) if E else None, _ptr(W2), RADIAL_HIDDEN,
                                           float(scale), int(pad_node), _ptr(m), _dtype(x, *((y,) if E else ())),
                                           _stream(stream)))
    return m


def conv_backward_radial(t: Table, csc, x, y, h, W2, dm, scale: float, out=None, stream=None, pad_node: int = -1):
    """Returns (dx, dy, dh): conv_backward with dw folded into dh = sum_{p,q} W2 dw (dw never stored)."""
    import torch
    cp, ce, cr = csc
    _contig(x, y, h, W2, dm)
    N, E = x.shape[0], y.shape[0]
    _csc_shapes(csc, N, E)
    _shape("x", x, N, t.d1, t.mul)
    _shape("y", y, E, t.d2)
    _radial_operands(t, E, h, W2)
    _shape("dm", dm, N, t.D, t.mul)
    if out is None:
        f = dict(dtype=torch.float32)
        out = (torch.empty_like(x, **f), torch.empty_like(y, **f), torch.empty_like(h, **f))
    dx, dy, dh = out
    _shape("dx", dx, N, t.d1, t.mul)
    _shape("dy", dy, E, t.d2)
    _shape("dh", dh, E, RADIAL_HIDDEN)
    _f32_out(dx, dy, dh, h, W2)
    _check(load().e3gb_conv_backward_radial(t.handle, N, E, _ptr(cp), _ptr(ce) if E else None,
                                            _ptr(cr) if E else None, _ptr(x), _ptr(y) if E else None,
                                            _ptr(h) if E else None, _ptr(W2), RADIAL_HIDDEN, _ptr(dm), float(scale),
                                            int(pad_node), _ptr(dx), _ptr(dy) if E else None,
                                            _ptr(dh) if E else None, _dtype(x, dm, *((y,) if E else ())),
                                            _stream(stream)))
    return dx, dy, dh


def conv_double_backward(t: Table, rowptr, sender, csc, x, y, w, dm, delta_dx, delta_dy, delta_dw, scale: float,
                         out=None, stream=None, pad_node: int = -1):
    """Eq. (17)-(18): returns (delta_x, delta_y, delta_w, delta_dm), the gradient of
    <dx, delta_dx> + <dy, delta_dy> + <dw, delta_dw> over (x, y, w, dm)."""
    import torch
    cp, ce, cr = csc
    _contig(rowptr, sender, x, y, w, dm, delta_dx, delta_dy, delta_dw)
    N, E = x.shape[0], y.shape[0]
    _shape("rowptr", rowptr, N + 1)
    _shape("sender", sender, E)
    _csc_shapes(csc, N, E)
    _conv_operands(t, N, E, x, y, w)
    _conv_operands(t, N, E, delta_dx, delta_dy, delta_dw, ("delta_dx", "delta_dy", "delta_dw"))
    _shape("dm", dm, N, t.D, t.mul)
    if out is None:
        f = dict(dtype=torch.float32)
        out = (torch.empty_like(x, **f), torch.empty_like(y, **f), torch.empty_like(w, **f),
               torch.empty_like(dm, **f))
    gx, gy, gw, gdm = out
    _conv_operands(t, N, E, gx, gy, gw, ("delta_x", "delta_y", "delta_w"))
    _shape("delta_dm", gdm, N, t.D, t.mul)
    _f32_out(gx, gy, gw, gdm)
    e = (lambda a: _ptr(a) if E else None)
    _check(load().e3gb_conv_double_backward(
        t.handle, N, E, _ptr(rowptr), e(sender), _ptr(cp), e(ce), e(cr), _ptr(x), e(y), e(w), _ptr(dm),
        _ptr(delta_dx), e(delta_dy), e(delta_dw), float(scale), int(pad_node), _ptr(gx), e(gy), e(gw), _ptr(gdm),
        _dtype(x, dm, delta_dx, *((y, w, delta_dy, delta_dw) if E else ())), _stream(stream)))
    return gx, gy, gw, gdm


def coo_tp_forward(rec, coef, x, y, w, D: int, out=None, stream=None):
    """Tensor product with runtime COO coefficients: rec int32 [n,4] (i0, i1, i2, path) and
    coef fp32 [n] on the device; x [R,d1,mul], y [R,d2], w [R,P,mul] -> z [R,D,mul] fp32."""
    import torch
    _contig(rec, coef, x, y, w)
    R, d1, mul = x.shape
    z = out if out is not None else torch.empty((R, D, mul), dtype=torch.float32, device=x.device)
    _f32_out(z)
    n = rec.shape[0]
    _check(load().e3gb_coo_tp_forward(R, d1, y.shape[1], D, w.shape[1], mul, n, _ptr(rec) if n else None,
                                      _ptr(coef) if n else None, _ptr(x), _ptr(y), _ptr(w), _ptr(z), _dtype(x, y, w),
                                      _stream(stream)))
    return z


def coo_tp_backward(rec, coef, x, y, w, dz, out=None, stream=None):
    """(dx, dy, dw) of coo_tp_forward."""
    import torch
    _contig(rec, coef, x, y, w, dz)
    R, d1, mul = x.shape
    if out is None:
        f = dict(dtype=torch.float32)
        out = (torch.empty_like(x, **f), torch.empty_like(y, **f), torch.empty_like(w, **f))
    dx, dy, dw = out
    _f32_out(dx, dy, dw)
    n = rec.shape[0]
    _check(load().e3gb_coo_tp_backward(R, d1, y.shape[1], dz.shape[1], w.shape[1], mul, n, _ptr(rec) if n else None,
                                       _ptr(coef) if n else None, _ptr(x), _ptr(y), _ptr(w), _ptr(dz), _ptr(dx),
                                       _ptr(dy), _ptr(dw), _dtype(x, y, w, dz), _stream(stream)))
    return dx, dy, dw


def _dtype_code(name, t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _elsewhere(name, t, at):
    where = "host memory" if at < 0 else f"cuda:{at}"
    raise ValueError(f"{name} is on {t.device}, expected all tensors of a call in the same place ({where})")


def _f32_param(name, t, at, *shape):
    """The address of a contiguous float32 parameter, gradient or statistics array of that shape
    (None for None) on device number `at` (-1: the host)."""
    import torch
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.get_device() != at:
        _elsewhere(name, t, at)
    if t.shape != shape:
        _shape(name, t, *shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _current(device):
    """The current stream, raw, of the tensors' device, which has to be the current one: launches go there."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}: expected device memory")
    here = torch._C._cuda_getDevice()
    if device.index != here:
        raise ValueError(f"tensors on {device}, but the current device is cuda:{here}")
    return torch._C._cuda_getCurrentRawStream(here)


def _on(stream, call, *args, out=None):
    """call(*args) with `stream` as the current one. What the call allocates then belongs to that stream (memory
    that went back to the caller's stream may still be in use there), and the results are kept from reuse until
    the caller's stream is done with them too."""
    import torch
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        results = call(*args)
    for t in results:
        if t is not None and t is not out:
            t.record_stream(caller)
    return results


def _apart(params, copies, moments):
    """Refuses contiguous tensors of which two share memory: a step writes all of them at once. moments: [(name,
    tensor)]."""
    tensors = [*params, *copies, *(t for _, t in moments)]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.nbytes, k) for k, t in enumerate(tensors) if t is not None and t.numel())
    n = len(params)
    name = lambda k: (f"params[{k}]" if k < n else f"copies[{k - n}]" if k < 2 * n else moments[k - 2 * n][0])  # noqa: E731
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError(f"{name(a)} and {name(b)} share memory")


def _written(*tensors):
    """Raises the version counters of tensors that a call wrote by their addresses, so that autograd refuses a
    backward pass that had saved one of them."""
    import torch
    torch.autograd.graph.increment_version([t for t in tensors if t is not None and not t.is_inference()])


def _row_stride(name, t, at, R, C):
    """Entries between the rows of t [R, C], whose rows are contiguous and do not overlap, on device `at`."""
    if t.get_device() != at:
        _elsewhere(name, t, at)
    if t.shape != (R, C):
        _shape(name, t, R, C)
    s0, s1 = t.stride()
    if (s1 != 1 and C > 1) or (s0 < C and R > 1):
        raise ValueError(f"{name}: strides {(s0, s1)}: rows must be contiguous and must not overlap")
    return s0 if R > 1 else C


def _given_workspace(ws, at):
    if ws.get_device() != at:
        _elsewhere("workspace", ws, at)
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws


@lru_cache(maxsize=256)
def _layer_norm_workspace(R, C):
    return max(16, load().e3gb_layer_norm_backward_workspace_bytes(R, C))


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, out=None, dtype=None, stream=None):
    """(y, stats): y [R, C] = (x - mean) * rstd * weight + bias for every row of x [R, C], whose
    rows may be strided (x[:, 0, :] of [N, d1, mul] features needs no copy); stats [R, 2] = (mean,
    rstd), which the backward takes. weight, bias: float32 [C] or None. x: float32 or bfloat16; y:
    float32, or `dtype`."""
    import torch
    if stream is not None:
        return _on(stream, layer_norm_forward, x, weight, bias, eps, out, dtype, out=out)
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (rows, channels)")
    (R, C), dev, at, f = x.shape, x.device, x.get_device(), torch.float32
    xs, w, b = _row_stride("x", x, at, R, C), _f32_param("weight", weight, at, C), _f32_param("bias", bias, at, C)
    y = torch.empty((R, C), dtype=dtype or f, device=dev) if out is None else out
    ys = C if out is None else _row_stride("y", out, at, R, C)
    xd, yd = _dtype_code("x", x), _dtype_code("y", y)
    stats = torch.empty((R, 2), dtype=f, device=dev)
    _check((_lib or load()).e3gb_layer_norm_forward(R, C, x.data_ptr(), xs, xd, w, b, eps, y.data_ptr(), ys, yd,
                                                    stats.data_ptr(), _current(dev)))
    if out is not None:
        _written(out)
    return y, stats


def layer_norm_backward(x, weight, stats, dy, out=None, dtype=None, params: bool = True, workspace=None, stream=None):
    """(dx, dweight, dbias) of layer_norm_forward for the cotangent dy [R, C] and the forward's
    stats. dx: float32, or `dtype`; dweight, dbias: float32 [C] (with params=False: None, and only dx
    is computed)."""
    import torch
    if stream is not None:
        return _on(stream, layer_norm_backward, x, weight, stats, dy, out, dtype, params, workspace, out=out)
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (rows, channels)")
    (R, C), dev, at, f = x.shape, x.device, x.get_device(), torch.float32
    xs, dys = _row_stride("x", x, at, R, C), _row_stride("dy", dy, at, R, C)
    w, st = _f32_param("weight", weight, at, C), _f32_param("stats", stats, at, R, 2)
    dx = torch.empty((R, C), dtype=dtype or f, device=dev) if out is None else out
    dxs = C if out is None else _row_stride("dx", out, at, R, C)
    xd, dyd, dxd = _dtype_code("x", x), _dtype_code("dy", dy), _dtype_code("dx", dx)
    dw = db = ws = None
    pw = pb = pws = nws = 0
    if params:
        dw, db = torch.empty(C, dtype=f, device=dev), torch.empty(C, dtype=f, device=dev)
        if workspace is None:
            ws = torch.empty(_layer_norm_workspace(R, C), dtype=torch.uint8, device=dev)
        else:
            ws = _given_workspace(workspace, at)
        pw, pb, pws, nws = dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size()
    _check((_lib or load()).e3gb_layer_norm_backward(R, C, x.data_ptr(), xs, xd, w, st, dy.data_ptr(), dys, dyd,
                                                     dx.data_ptr(), dxs, dxd, pw, pb, pws, nws, _current(dev)))
    if out is not None:
        _written(out)
    return dx, dw, db


@lru_cache(maxsize=64)
def _irreps_of(blocks: tuple, mul: int):
    """(reference to the C irreps, rows, number of even scalar blocks)."""
    n = len(blocks)
    ints = ctypes.c_int32 * max(1, n)
    ir = _Irreps(n, ints(*[b[0] for b in blocks]), ints(*[b[1] for b in blocks]), mul)
    return ctypes.byref(ir), sum(2 * l + 1 for l, _ in blocks), sum(1 for l, p in blocks if l == 0 and p == 1)


@lru_cache(maxsize=256)
def _irreps_norm_workspace(blocks: tuple, mul: int, N: int):
    return max(16, load().e3gb_irreps_norm_backward_workspace_bytes(_irreps_of(blocks, mul)[0], N))


def _irreps_operand(blocks, x):
    """(blocks as a key, the C irreps, even scalar blocks) for x [N, d1, mul]."""
    key = tuple(map(tuple, blocks))
    if x.dim() != 3:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (nodes, rows, mul)")
    ir, d1, scalars = _irreps_of(key, x.shape[2])
    if x.shape[1] != d1:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (nodes, {d1}, mul)")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    return key, ir, scalars


def _same_layout(name, t, x):
    if t.get_device() != x.get_device():
        _elsewhere(name, t, x.get_device())
    if t.shape != x.shape:
        _shape(name, t, *x.shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def irreps_norm_forward(blocks, x, weight=None, bias=None, eps: float = 1e-5, out=None, dtype=None, stream=None):
    """(y, stats): the norm of irreps features x [N, d1, mul], blocks [(l, parity)] (as in
    Table.create; any mul). Every (node, block) is scaled by one number, 1/rms of its entries, then
    per channel by weight [n_blocks, mul]; even scalars lose their mean over the channels first and
    take bias [number of even scalar blocks, mul]. Rotations and reflections commute with it. stats
    [N, n_blocks, 2] = (mean or 0, 1/rms) goes to the backward. y: float32, or `dtype`."""
    import torch
    if stream is not None:
        return _on(stream, irreps_norm_forward, blocks, x, weight, bias, eps, out, dtype, out=out)
    _, ir, scalars = _irreps_operand(blocks, x)
    shape, nb, dev, at, f = x.shape, len(blocks), x.device, x.get_device(), torch.float32
    N, _, mul = shape
    w, b = _f32_param("weight", weight, at, nb, mul), _f32_param("bias", bias, at, scalars, mul)
    y = torch.empty(shape, dtype=dtype or f, device=dev) if out is None else out
    if out is not None:
        _same_layout("y", y, x)
    xd, yd = _dtype_code("x", x), _dtype_code("y", y)
    stats = torch.empty((N, nb, 2), dtype=f, device=dev)
    _check((_lib or load()).e3gb_irreps_norm_forward(ir, N, x.data_ptr(), xd, w, b if scalars else None, eps, y.data_ptr(),
                                                     yd, stats.data_ptr(), _current(dev)))
    if out is not None:
        _written(out)
    return y, stats


def irreps_norm_backward(blocks, x, weight, stats, dy, out=None, dtype=None, params: bool = True, workspace=None,
                         stream=None):
    """(dx, dweight, dbias) of irreps_norm_forward for the cotangent dy [N, d1, mul] and the
    forward's stats; dbias is None where there is no even scalar block. params=False: dx only."""
    import torch
    if stream is not None:
        return _on(stream, irreps_norm_backward, blocks, x, weight, stats, dy, out, dtype, params, workspace, out=out)
    key, ir, scalars = _irreps_operand(blocks, x)
    shape, nb, dev, at, f = x.shape, len(key), x.device, x.get_device(), torch.float32
    N, _, mul = shape
    w, st = _f32_param("weight", weight, at, nb, mul), _f32_param("stats", stats, at, N, nb, 2)
    _same_layout("dy", dy, x)
    dx = torch.empty(shape, dtype=dtype or f, device=dev) if out is None else out
    if out is not None:
        _same_layout("dx", dx, x)
    xd, dyd, dxd = _dtype_code("x", x), _dtype_code("dy", dy), _dtype_code("dx", dx)
    dw = db = ws = None
    pw = pb = pws = nws = 0
    if params:
        dw = torch.empty((nb, mul), dtype=f, device=dev)
        if workspace is None:
            ws = torch.empty(_irreps_norm_workspace(key, mul, N), dtype=torch.uint8, device=dev)
        else:
            ws = _given_workspace(workspace, at)
        pw, pws, nws = dw.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size()
        if scalars:
            db = torch.empty((scalars, mul), dtype=f, device=dev)
            pb = db.data_ptr()
    _check((_lib or load()).e3gb_irreps_norm_backward(ir, N, x.data_ptr(), xd, w, st, dy.data_ptr(), dyd, dx.data_ptr(), dxd,
                                                      pw, pb, pws, nws, _current(dev)))
    if out is not None:
        _written(out)
    return dx, dw, db


_GET_DTYPE = attrgetter("dtype")
_MOMENTS = ("m", "v", "m_scale", "v_scale")


@dataclass
class AdamW:
    """AdamW handle (e3gb_adamw) over float32 parameters, which it updates where they lie: they must
    keep their storage while the handle lives. m, v: the moments of all tensors in one buffer each,
    tensor i's from entry starts[i]; float32, or with state_bits=8 float8_e4m3fn and float8_e5m2 with a
    power-of-two scale (m_scale, v_scale) for each 256 entries: saved and restored as any tensors, also by
    setting one of the four attributes (to a tensor of the same type, shape and device)."""
    handle: ctypes.c_void_p
    params: tuple
    numel: tuple
    copies: tuple
    state_bits: int
    seed: int
    starts: list
    m: object
    v: object
    m_scale: object
    v_scale: object
    plan: object
    workspace: object
    streams: set = field(default_factory=set)   # raw, on which the buffers are known to be in use
    tracked: list = field(default_factory=list)   # tensors whose version counters a step raises
    given: tuple = ()                             # the parameters and copies as create() got them
    kinds: dict | None = None                     # shape and type of each moment, once create() is done

    @classmethod
    def create(cls, params, weight_decay=0.01, state_bits: int = 32, state=None, copies=None, seed: int = 0) -> "AdamW":
        """params: contiguous float32 device tensors. weight_decay: one number, or one for each
        tensor. state: (m, v) or (m, v, m_scale, v_scale) to use as the moments (zeros by default).
        copies: bfloat16 tensors (or None) that every step also writes the rounded parameters to.
        seed: of the bits that round 8-bit moments. No two of all these may share memory."""
        import torch
        params = tuple(params)
        n = len(params)
        copies = (None,) * n if copies is None else tuple(copies)
        given = tuple(t for t in params + copies if t is not None)
        params, copies = tuple(p.detach() for p in params), tuple(c if c is None else c.detach() for c in copies)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
        if n < 1 or len(copies) != n or len(decay) != n:
            raise ValueError(f"{n} parameters, {len(copies)} copies, {len(decay)} weight decays")
        if not 0 <= seed < 1 << 32:
            raise ValueError("seed must fit in 32 bits")
        at = params[0].get_device()
        for i, (p, c) in enumerate(zip(params, copies)):
            _f32_param(f"params[{i}]", p, at, *p.shape)
            if c is not None:
                if c.dtype != torch.bfloat16:
                    raise TypeError(f"copies[{i}] must be bfloat16")
                if c.get_device() != at:
                    _elsewhere(f"copies[{i}]", c, at)
                _shape(f"copies[{i}]", c, *p.shape)
                _contig(c)
        moments = list(zip(_MOMENTS, state or ()))
        for name, t in moments:
            if t.get_device() != at:
                _elsewhere(name, t, at)
            _contig(t)
        _apart(params, copies, moments)
        lib = load()
        ptrs = lambda ts: (ctypes.c_void_p * n)(*[None if t is None else t.data_ptr() for t in ts])  # noqa: E731
        h = ctypes.c_void_p()
        _check(lib.e3gb_adamw_create(n, (ctypes.c_int64 * n)(*[p.numel() for p in params]), ptrs(params), ptrs(copies),
                                     (ctypes.c_float * n)(*decay), state_bits, ctypes.byref(h)))
        a = cls(h, params, tuple(p.numel() for p in params), copies, state_bits, seed, [], None, None, None, None, None, None)
        entries, plan_bytes, ws_bytes = ctypes.c_int64(), ctypes.c_size_t(), ctypes.c_size_t()
        starts = (ctypes.c_int64 * n)()
        _check(lib.e3gb_adamw_info(h, ctypes.byref(entries), ctypes.byref(plan_bytes), ctypes.byref(ws_bytes), starts))
        a.starts, dev, E = list(starts), params[0].device, entries.value
        host = torch.empty(plan_bytes.value, dtype=torch.uint8)
        _check(lib.e3gb_adamw_plan(h, host.data_ptr()))
        a.plan = host.to(dev)
        a.workspace = torch.empty(ws_bytes.value, dtype=torch.uint8, device=dev)
        eight = state_bits == 8
        want = [((E,), torch.float8_e4m3fn if eight else torch.float32), ((E,), torch.float8_e5m2 if eight else torch.float32)]
        want += [((E // 256,), torch.float32)] * (2 if eight else 0)
        if state is None:
            state = [torch.zeros(s, dtype=torch.uint8 if eight and d != torch.float32 else d, device=dev).view(d)
                     for s, d in want]
        if len(state) != len(want):
            raise ValueError(f"state of {len(state)} tensors, expected {len(want)}")
        kinds = dict(zip(_MOMENTS, want))
        for name, t in zip(_MOMENTS, state):
            a._fits(name, t, kinds)
            setattr(a, name, t)
        a.given, a.kinds = given, kinds
        a._track()
        if dev.type == "cuda":
            here = torch.cuda.current_stream(dev)
            here.synchronize()                  # the first step may be on any stream
            a.streams = {here.cuda_stream}      # what was allocated here needs no mark for it
        return a

    def __setattr__(self, name, value):
        if name not in _MOMENTS or self.kinds is None:
            return object.__setattr__(self, name, value)
        self._fits(name, value, self.kinds)
        others = [(k, t) for k, t in self._moments() if k != name]
        _apart(self.params, self.copies, others + [(name, value)])
        object.__setattr__(self, name, value)
        self.streams = set()
        self._track()

    def _moments(self):
        return [(k, getattr(self, k)) for k in _MOMENTS if getattr(self, k) is not None]

    def _fits(self, name, t, kinds):
        if name not in kinds:
            raise ValueError(f"moments of {self.state_bits} bits have no {name}")
        shape, dtype = kinds[name]
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.get_device() != self.plan.get_device():
            _elsewhere(name, t, self.plan.get_device())
        _shape(name, t, *shape)
        _contig(t)

    def _track(self):
        """Views of one buffer share its version counter."""
        held = [*self.given, *(t for _, t in self._moments())]
        counted = {id(b): b for b in (t if t._base is None else t._base for t in held)}
        self.tracked = [t for t in counted.values() if not t.is_inference()]

    def keep_for(self, raw: int):
        """Marks every buffer that the kernels read or write as used on the current stream (raw): a step may still
        be queued there when the handle, perhaps the last holder of all of them, goes away."""
        import torch
        s = torch.cuda.current_stream(self.plan.device)
        for t in (self.plan, self.workspace, self.m, self.v, self.m_scale, self.v_scale, *self.params, *self.copies):
            if t is not None:
                t.record_stream(s)
        self.streams.add(raw)

    def gradient_addresses(self, grads):
        """(dtype code, array of addresses, 0 for None, whether there is no None) of one step's gradients, checked
        against the parameters. With hundreds of tensors this is most of a step's time on the host, so the checks
        run as maps over the whole list; the loop below finds out what is wrong, or skips None."""
        import torch
        T, n = torch.Tensor, len(self.params)
        if len(grads) != n:
            raise ValueError(f"{len(grads)} gradients, {n} parameters")
        codes = {torch.float32: F32, torch.bfloat16: BF16}
        try:
            kinds = set(map(_GET_DTYPE, grads))
            if (len(kinds) == 1 and tuple(map(T.numel, grads)) == self.numel and all(map(T.is_contiguous, grads))
                    and set(map(T.get_device, grads)) == {self.plan.get_device()}):
                kind = kinds.pop()
                if kind in codes:
                    return codes[kind], array.array("Q", map(T.data_ptr, grads)), True
        except (AttributeError, TypeError):
            pass                                   # a None among them
        kind, out = None, array.array("Q", bytes(8 * n))
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if g is None:
                continue
            kind = g.dtype if kind is None else kind
            if g.dtype not in codes:
                raise TypeError(f"grads[{i}] must be float32 or bfloat16, got {g.dtype}")
            if g.dtype != kind:
                raise TypeError(f"gradients must all be float32 or all bfloat16: grads[{i}] is {g.dtype}")
            if g.numel() != p.numel() or g.device != p.device:
                raise ValueError(f"grads[{i}]: {tuple(g.shape)} on {g.device}, expected {tuple(p.shape)} on {p.device}")
            if not g.is_contiguous():
                raise ValueError(f"grads[{i}] must be contiguous")
            out[i] = g.data_ptr()
        return codes.get(kind, F32), out, not any(g is None for g in grads)

    def moments(self, i: int):
        """(m, v) of tensor i as float32 tensors of its shape."""
        p = self.params[i]
        s, n = self.starts[i], p.numel()
        out = []
        for t, scale in ((self.m, self.m_scale), (self.v, self.v_scale)):
            if scale is None:
                out.append(t[s:s + n].view(p.shape).clone())
            else:
                e = -(-n // 256) * 256
                x = t[s:s + e].float().view(-1, 256) * scale[s // 256:(s + e) // 256, None]
                out.append(x.reshape(-1)[:n].view(p.shape))
        return tuple(out)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.e3gb_adamw_destroy(h)
            self.handle = None


def adamw_step(opt: AdamW, grads, lr: float, step: int, betas=(0.9, 0.999), eps: float = 1e-8, max_norm=None,
               stream=None):
    """One AdamW step (the step-th, from 1) on opt's parameters with grads: one tensor for each
    parameter, all float32 or all bfloat16, contiguous, of its size; None leaves a parameter as it is.
    max_norm: scale the gradients so that the 2-norm of all of them is at most that; the norm before
    scaling is returned ([1] float32 on the device, else None), and a step whose norm is not finite
    changes nothing."""
    import torch
    if stream is not None:
        return _on(stream, lambda: (adamw_step(opt, grads, lr, step, betas, eps, max_norm),))[0]
    code, addresses, every = opt.gradient_addresses(grads)
    if max_norm is not None and not max_norm > 0:
        raise ValueError("max_norm must be positive")
    dev = opt.plan.device
    norm = None if max_norm is None else torch.empty(1, dtype=torch.float32, device=dev)
    rates = _AdamwRates(lr, betas[0], betas[1], eps, max_norm or 0.0, step, opt.seed)
    s, ms, vs = _current(dev), opt.m_scale, opt.v_scale
    if s not in opt.streams:
        opt.keep_for(s)
    _check(_lib.e3gb_adamw_step(opt.handle, opt.plan.data_ptr(), addresses.buffer_info()[0], code, opt.m.data_ptr(), opt.v.data_ptr(),
                                None if ms is None else ms.data_ptr(), None if vs is None else vs.data_ptr(),
                                ctypes.byref(rates), None if norm is None else norm.data_ptr(),
                                opt.workspace.data_ptr(), opt.workspace.numel(), s))
    if every:
        torch.autograd.graph.increment_version(opt.tracked)
    else:
        given = [i for i, g in enumerate(grads) if g is not None]
        _written(*(opt.params[i] for i in given), *(opt.copies[i] for i in given), opt.m, opt.v, ms, vs)
    return norm


def check_device_status(stream=None) -> int:
    """Synchronise and read/clear the device error word; raises E3GBError if it was set."""
    flags = ctypes.c_int32()
    st = load().e3gb_check_device_status(_stream(stream), ctypes.byref(flags))
    if st != OK:
        raise E3GBError(st, load().e3gb_last_error().decode())
    return flags.value


def shard_graphs(graph_ptr, rowptr, sender, world: int, rank: int) -> tuple[int, int, int, int]:
    """Data-parallel split of a batch of independent graphs (molecules) stored as one
    receiver-sorted CSR: graph g owns nodes [graph_ptr[g], graph_ptr[g+1]) and every edge into
    them, and each of its edges must come from one of its own nodes. Returns (n0, n1, e0, e1):
    rank's contiguous run of whole graphs, cut at the graph boundaries nearest to r * E / world
    so that the ranks' edge counts differ by at most about one graph's edges. The rank's own
    CSR is rowptr[n0:n1+1] - e0 with senders sender[e0:e1] - n0; no edge crosses ranks, so
    the ranks exchange nothing on the data path (host logic, numpy; raises ValueError if an
    edge leaves its graph)."""
    import numpy as np

    gp = np.asarray(graph_ptr, dtype=np.int64)
    rp = np.asarray(rowptr, dtype=np.int64)
    sd = np.asarray(sender, dtype=np.int64)
    if world < 1 or not 0 <= rank < world:
        raise ValueError(f"rank {rank} outside world {world}")
    N, E = rp.shape[0] - 1, int(rp[-1]) if rp.shape[0] else 0
    if gp.ndim != 1 or gp.shape[0] < 1 or gp[0] != 0 or gp[-1] != N or np.any(np.diff(gp) < 0):
        raise ValueError("graph_ptr must rise from 0 to the node count")
    if rp[0] != 0 or np.any(np.diff(rp) < 0) or sd.shape[0] != E:
        raise ValueError("rowptr / sender do not form a CSR")
    # the graph of each edge's receiver and of its sender must agree
    recv = np.repeat(np.arange(N, dtype=np.int64), np.diff(rp))
    g_of = lambda v: np.searchsorted(gp, v, side="right") - 1
    if E and (np.any(sd < 0) or np.any(sd >= N) or np.any(g_of(recv) != g_of(sd))):
        raise ValueError("an edge joins two graphs: the batch cannot be split without a halo")
    eb = rp[gp]   # edge offset at each graph boundary (non-decreasing)
    cut = [0]
    for r in range(1, world):
        t = r * E / world
        b = int(np.searchsorted(eb, t))
        if b > 0 and (b >= eb.shape[0] or t - eb[b - 1] <= eb[b] - t):
            b -= 1
        cut.append(max(b, cut[-1]))
    cut.append(gp.shape[0] - 1)
    n0, n1 = int(gp[cut[rank]]), int(gp[cut[rank + 1]])
    return n0, n1, int(rp[n0]), int(rp[n1])
