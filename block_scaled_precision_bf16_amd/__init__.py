"""Python binding of libmxcast (include/mxcast.h): block-scaled quantisation of
bf16 tensors on MI355X, and the products of what it writes.

Argument marshalling only.  Every step of the casts and products runs in the HIP kernels of
libmxcast.so; PyTorch provides device memory and the stream.  If the library
is not built, importing a function raises -- there is no fallback path.

The same names as the C ABI:
    mx_quantize, mx_quantize_workspace_size, mx_scale_size, mx_quantize_grouped,
    mx_quantize_grouped_workspace_size, mx_grouped_scale_size, mx_quantize_gated,
    mx_fused_values, mx_absmax_bf16, nvfp4_quantize_transpose,
    mx_matmul, mx_matmul_grouped, mx_matmul_wgrad_grouped, their
    *_workspace_size, nvfp4_matvec, nvfp4_matvec_experts, mx_rmsnorm,
    mx_rmsnorm_backward, moe_route, moe_route_backward, moe_sort, moe_gather,
    moe_combine, moe_combine_backward, mx_status_str, mx_abi_version
take torch tensors (bf16 inputs, or int16/uint16 holding bf16 bits, on a ROCm
device).  The casts return dicts of uint8 / float32 torch tensors on the same
device; the products take those and return a bf16 or float32 tensor.
The MXFP8 casts take the format flags ELEM_E5M2 / SCALE_ROUND_UP and the
layout flag SCALE_TILED OR-ed into `axis`, as the C ABI does.
`lib()` returns the raw ctypes library for callers that pass pointers
themselves.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxcast.so")

ROWWISE, COLWISE = 1, 2
ELEM_E5M2, SCALE_ROUND_UP = 4, 8     # MXFP8 format flags, OR-ed into axis
SCALE_TILED = 16                     # GEMM-ready scale layout flag, OR-ed into axis
FUSE_NONE, FUSE_GELU, FUSE_DGELU, FUSE_DSILU, FUSE_DBIAS = 0, 1, 2, 3, 0x10
GATED_SWIGLU, GATED_GEGLU = 1, 2
OP_GATED, OP_DGATED = 0x100, 0x200
# flags of the products (with SCALE_TILED): operand formats, output type
A_E5M2, B_E5M2, OUT_F32, ACCUMULATE = 4, 32, 64, 128
# flags of the router (its logits' type, ROUTE_F32 in the C ABI, comes from the tensor)
ROUTE_SIGMOID, ROUTE_RENORM, ROUTE_GROUP_PAIR, _ROUTE_F32 = 1, 2, 4, 8
(MX_OK, MX_ERR_NULL, MX_ERR_ENUM, MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_WORKSPACE,
 MX_ERR_ALIAS, MX_ERR_HIP, MX_ERR_UNSUPPORTED) = range(9)

EXPORTS = ("mx_quantize", "mx_quantize_workspace_size", "mx_quantize_noalloc", "mx_scale_size", "mx_quantize_grouped",
           "mx_quantize_grouped_workspace_size", "mx_grouped_scale_size", "mx_quantize_gated",
           "mx_quantize_gated_grouped", "mx_quantize_dgated_grouped",
           "mx_quantize_dgated", "mx_fused_values",
           "mx_absmax_bf16", "nvfp4_quantize_transpose", "nvfp4_quantize_transpose_2d",
           "mx_absmax_bf16_grouped", "nvfp4_quantize_transpose_grouped",
           "mx_matmul", "mx_matmul_grouped", "mx_matmul_wgrad_grouped",
           "mx_matmul_workspace_size", "mx_matmul_grouped_workspace_size",
           "mx_matmul_wgrad_grouped_workspace_size", "nvfp4_matvec", "nvfp4_matvec_experts",
           "mx_rmsnorm", "mx_rmsnorm_workspace_size", "mx_rmsnorm_backward", "mx_rmsnorm_backward_workspace_size",
           "moe_route", "moe_route_backward", "moe_sort", "moe_sort_rows", "moe_sort_workspace_size",
           "moe_gather", "moe_combine", "moe_combine_backward",
           "mx_status_str", "mx_abi_version")


class MxError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {mx_status_str(status)} (status {status})")


_lib = None
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


def lib():
    """The loaded libmxcast.so with argument types set (raises if not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                              "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        L.mx_quantize.restype = ctypes.c_int
        L.mx_quantize.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_uint, ctypes.c_int,
                                  _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.mx_quantize_noalloc.restype = ctypes.c_int
        L.mx_quantize_noalloc.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_uint, ctypes.c_int,
                                          _vp, _vp, _vp, _vp, _vp, _vp]
        L.mx_quantize_workspace_size.restype = ctypes.c_size_t
        L.mx_quantize_workspace_size.argtypes = [_i64, _i64, ctypes.c_uint, ctypes.c_int]
        L.mx_scale_size.restype = ctypes.c_size_t
        L.mx_scale_size.argtypes = [_i64, _i64, ctypes.c_uint]
        L.mx_quantize_grouped.restype = ctypes.c_int
        L.mx_quantize_grouped.argtypes = [_vp, _vp, _i64, _vp, ctypes.c_int, ctypes.c_uint,
                                          ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                          ctypes.c_size_t, _vp]
        L.mx_quantize_grouped_workspace_size.restype = ctypes.c_size_t
        L.mx_quantize_grouped_workspace_size.argtypes = [_i64, _vp, ctypes.c_int, ctypes.c_uint,
                                                         ctypes.c_int]
        L.mx_grouped_scale_size.restype = ctypes.c_size_t
        L.mx_grouped_scale_size.argtypes = [_i64, _vp, ctypes.c_int, ctypes.c_uint, ctypes.c_int]
        L.mx_quantize_gated_grouped.restype = ctypes.c_int
        L.mx_quantize_gated_grouped.argtypes = [_vp, _i64, _vp, ctypes.c_int, ctypes.c_uint,
                                                ctypes.c_int, _vp, _vp, _vp, _vp, _vp]
        L.mx_quantize_dgated_grouped.restype = ctypes.c_int
        L.mx_quantize_dgated_grouped.argtypes = [_vp, _vp, _i64, _vp, ctypes.c_int, ctypes.c_uint,
                                                 ctypes.c_int, _vp, _vp, _vp, _vp, _vp]
        L.mx_quantize_gated.restype = ctypes.c_int
        L.mx_quantize_gated.argtypes = [_vp, _i64, _i64, ctypes.c_uint, ctypes.c_int,
                                        _vp, _vp, _vp, _vp, _vp]
        L.mx_quantize_dgated.restype = ctypes.c_int
        L.mx_quantize_dgated.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_uint, ctypes.c_int,
                                         _vp, _vp, _vp, _vp, _vp]
        L.mx_fused_values.restype = ctypes.c_int
        L.mx_fused_values.argtypes = [_vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp]
        L.mx_absmax_bf16.restype = ctypes.c_int
        L.mx_absmax_bf16.argtypes = [_vp, _i64, _vp, _vp]
        L.nvfp4_quantize_transpose.restype = ctypes.c_int
        L.nvfp4_quantize_transpose.argtypes = [_vp, _i64, _i64, _vp, ctypes.c_uint,
                                               _vp, _vp, _vp, _vp, _vp, _vp]
        L.nvfp4_quantize_transpose_2d.restype = ctypes.c_int
        L.nvfp4_quantize_transpose_2d.argtypes = L.nvfp4_quantize_transpose.argtypes
        L.mx_absmax_bf16_grouped.restype = ctypes.c_int
        L.mx_absmax_bf16_grouped.argtypes = [_vp, _i64, _vp, ctypes.c_int, _vp, _vp]
        L.nvfp4_quantize_transpose_grouped.restype = ctypes.c_int
        L.nvfp4_quantize_transpose_grouped.argtypes = [_vp, _i64, _vp, ctypes.c_int, _vp,
                                                       ctypes.c_int, ctypes.c_uint, _vp, _vp,
                                                       _vp, _vp, _vp, _vp]
        L.mx_matmul.restype = ctypes.c_int
        L.mx_matmul.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_uint, _vp, _vp,
                                ctypes.c_size_t, _vp]
        L.mx_matmul_grouped.restype = ctypes.c_int
        L.mx_matmul_grouped.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _vp, ctypes.c_int,
                                        ctypes.c_uint, _vp, _vp, ctypes.c_size_t, _vp]
        L.mx_matmul_wgrad_grouped.restype = ctypes.c_int
        L.mx_matmul_wgrad_grouped.argtypes = L.mx_matmul_grouped.argtypes
        L.mx_matmul_workspace_size.restype = ctypes.c_size_t
        L.mx_matmul_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_uint]
        for f in (L.mx_matmul_grouped_workspace_size, L.mx_matmul_wgrad_grouped_workspace_size):
            f.restype = ctypes.c_size_t
            f.argtypes = [_i64, _i64, _vp, ctypes.c_int, ctypes.c_uint]
        L.nvfp4_matvec.restype = ctypes.c_int
        L.nvfp4_matvec.argtypes = [_vp, _i64, _vp, _vp, _vp, _i64, _i64, ctypes.c_uint, _vp, _vp]
        L.nvfp4_matvec_experts.restype = ctypes.c_int
        L.nvfp4_matvec_experts.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, ctypes.c_int, _i64,
                                           _i64, ctypes.c_uint, _vp, _vp]
        u32, f32, sz = ctypes.c_uint, ctypes.c_float, ctypes.c_size_t
        for name, args in (
                ("mx_rmsnorm", [_vp] * 3 + [_i64, _i64, f32, u32] + [_vp] * 10 + [sz, _vp]),
                ("mx_rmsnorm_backward", [_vp] * 7 + [_i64, _i64] + [_vp] * 3 + [sz, _vp]),
                ("moe_route", [_vp] * 2 + [_i64] * 5 + [f32, u32] + [_vp] * 4),
                ("moe_route_backward", [_vp] * 4 + [_i64] * 3 + [f32, u32] + [_vp] * 2),
                ("moe_sort", [_vp] + [_i64] * 5 + [_vp] * 4 + [sz, _vp]),
                ("moe_gather", [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp]),
                ("moe_combine", [_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp]),
                ("moe_combine_backward", [_vp, _vp, _i64, _i64] + [_vp] * 3 + [_i64, _i64] + [_vp] * 3)):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = args
        L.mx_rmsnorm_workspace_size.restype = sz
        L.mx_rmsnorm_workspace_size.argtypes = [_i64, u32]
        L.mx_rmsnorm_backward_workspace_size.restype = sz
        L.mx_rmsnorm_backward_workspace_size.argtypes = [_i64, _i64]
        L.moe_sort_rows.restype = _i64
        L.moe_sort_rows.argtypes = [_i64] * 4
        L.moe_sort_workspace_size.restype = sz
        L.moe_sort_workspace_size.argtypes = [_i64] * 3
        L.mx_status_str.restype = ctypes.c_char_p
        L.mx_status_str.argtypes = [ctypes.c_int]
        L.mx_abi_version.restype = ctypes.c_int
        L.mx_abi_version.argtypes = []
        _lib = L
    return _lib


def mx_status_str(status: int) -> str:
    return lib().mx_status_str(int(status)).decode()


def mx_abi_version() -> int:
    return lib().mx_abi_version()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _bf16_bits(t):
    if t is None:
        return None
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"expected bf16 (or int16/uint16 bf16 bits), got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t


def _check(status, where):
    if status != MX_OK:
        raise MxError(status, where)


def _2d(t, name):
    """A bf16-bits input that must be a contiguous 2-D tensor."""
    t = _bf16_bits(t)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t


def _half_width(W, name):
    """N of a gated row [gate | linear] of W elements (W must be even)."""
    if W % 2:
        raise ValueError(f"{name}: a [gate | linear] row has an even number of columns, got {W}")
    return W // 2


def _want_shape(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _group_total(group_rows, M):
    if any(int(r) < 0 for r in group_rows):
        raise ValueError("group row counts must be non-negative")
    if sum(int(r) for r in group_rows) != M:
        raise ValueError(f"group row counts sum to {sum(int(r) for r in group_rows)}, "
                         f"but the input has {M} rows")


def _outputs(o, need, dev):
    """Allocate the outputs the caller did not pass and check those it did.
    need maps name -> (shape, dtype).  A passed tensor must be a contiguous
    tensor of that dtype on the input's device with exactly as many elements
    as the library writes."""
    o = dict(o or {})
    for k, (shape, dtype) in need.items():
        t = o.get(k)
        if t is None:
            o[k] = torch.empty(shape, dtype=dtype, device=dev)
            continue
        numel = 1
        for d in shape:
            numel *= int(d)
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"out[{k!r}] must be a tensor")
        if t.dtype != dtype or t.numel() != numel or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"out[{k!r}] must be a contiguous {dtype} tensor of {numel} elements "
                             f"on {dev}; got {t.dtype}, {t.numel()} elements on {t.device}"
                             f"{'' if t.is_contiguous() else ', not contiguous'}")
    return o


def _on_device(dev, *tensors):
    """Every tensor the library reads or writes lives on one ROCm device (a
    host pointer handed to a kernel would fault the GPU)."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a ROCm (cuda) device, got {dev}")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on {dev}; got one on {t.device}")


def _f32_vec(t, n, name, dev):
    """A float32 device vector of n elements (amax, global scales)."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() != n \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return t


U8, F32, I16 = torch.uint8, torch.float32, torch.int16


def mx_quantize_workspace_size(M: int, K: int, axis: int = ROWWISE | COLWISE,
                               fusion: int = FUSE_NONE) -> int:
    return lib().mx_quantize_workspace_size(M, K, axis, fusion)


def mx_scale_size(rows: int, cols: int, axis: int = ROWWISE | COLWISE) -> int:
    return lib().mx_scale_size(rows, cols, axis)


def _scale_shape(rows, cols, axis):
    """One direction's scale tensor: [rows][ceil(cols/32)], or flat in the tile
    layout."""
    if axis & SCALE_TILED:
        return (max(1, mx_scale_size(rows, cols, axis)),)
    return (rows, -(-cols // 32))


def _mx_need(M, K, axis):
    """Outputs of an MXFP8 cast of a quantised [M][K] tensor."""
    need = {}
    if axis & ROWWISE:
        need["q_row"] = ((M, K), U8)
        need["s_row"] = (_scale_shape(M, K, axis), U8)
    if axis & COLWISE:
        need["q_col"] = ((K, M), U8)
        need["s_col"] = (_scale_shape(K, M, axis), U8)
    return need


def _workspace(workspace, need_bytes, dev):
    if workspace is None:
        return torch.empty(max(need_bytes, 16), dtype=U8, device=dev)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() \
            or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace


def mx_quantize(x, grad=None, axis=ROWWISE | COLWISE, fusion=FUSE_NONE, out=None,
                workspace=None, stream=None):
    """MXFP8 cast of x[M][K].  Returns {q_row, s_row, q_col, s_col, dbias}
    (None where not requested).  `out` may hold preallocated outputs and
    `workspace` a preallocated device buffer (needed only with FUSE_DBIAS)."""
    x = _2d(x, "x")
    M, K = x.shape
    grad = _2d(grad, "grad") if (fusion & 0xF) in (FUSE_DGELU, FUSE_DSILU) else None
    _want_shape(grad, (M, K), "grad")
    dev = x.device
    need = _mx_need(M, K, axis)
    if fusion & FUSE_DBIAS:
        need["dbias"] = ((K,), F32)
    o = _outputs(out, need, dev)
    ws_bytes = 0
    if fusion & FUSE_DBIAS:
        workspace = _workspace(workspace, mx_quantize_workspace_size(M, K, axis, fusion), dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    _on_device(dev, grad, *o.values(), workspace if fusion & FUSE_DBIAS else None)
    st = lib().mx_quantize(_ptr(x), _ptr(grad), M, K, axis, fusion,
                           _ptr(o.get("q_row")), _ptr(o.get("s_row")), _ptr(o.get("q_col")),
                           _ptr(o.get("s_col")), _ptr(o.get("dbias")),
                           _ptr(workspace) if fusion & FUSE_DBIAS else None, ws_bytes,
                           _stream(dev, stream))
    _check(st, "mx_quantize")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col", "dbias")}


NOALLOC_SCRATCH_BYTES = 4 << 20     # MX_NOALLOC_SCRATCH_BYTES


def mx_quantize_noalloc(x, out, grad=None, axis=ROWWISE | COLWISE, fusion=FUSE_NONE,
                        stream=None):
    """mx_quantize without any device allocation: `out` must hold every
    requested output (q_row, s_row, q_col, s_col, and dbias with FUSE_DBIAS)
    preallocated; dbias partials use the library's static device scratch
    (calls with FUSE_DBIAS that overlap on one GPU race; see mxcast.h)."""
    x = _2d(x, "x")
    M, K = x.shape
    grad = _2d(grad, "grad") if (fusion & 0xF) in (FUSE_DGELU, FUSE_DSILU) else None
    _want_shape(grad, (M, K), "grad")
    dev = x.device
    need = _mx_need(M, K, axis)
    if fusion & FUSE_DBIAS:
        need["dbias"] = ((K,), F32)
    missing = [k for k in need if (out or {}).get(k) is None]
    if missing:
        raise ValueError(f"mx_quantize_noalloc allocates nothing: out must hold {missing}")
    o = _outputs(out, need, dev)
    _on_device(dev, grad, *o.values())
    st = lib().mx_quantize_noalloc(_ptr(x), _ptr(grad), M, K, axis, fusion,
                                   _ptr(o.get("q_row")), _ptr(o.get("s_row")),
                                   _ptr(o.get("q_col")), _ptr(o.get("s_col")),
                                   _ptr(o.get("dbias")), _stream(dev, stream))
    _check(st, "mx_quantize_noalloc")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col", "dbias")}


def _rows_arg(group_rows):
    """Host int64 array of group row counts (kept alive by the caller)."""
    return (ctypes.c_int64 * len(group_rows))(*[int(r) for r in group_rows])


def mx_quantize_grouped_workspace_size(K: int, group_rows, axis: int = ROWWISE | COLWISE,
                                       fusion: int = FUSE_NONE) -> int:
    rows = _rows_arg(group_rows)
    return lib().mx_quantize_grouped_workspace_size(K, ctypes.cast(rows, _vp), len(group_rows),
                                                    axis, fusion)


def mx_grouped_scale_size(K: int, group_rows, axis: int, colwise: bool) -> int:
    rows = _rows_arg(group_rows)
    return lib().mx_grouped_scale_size(K, ctypes.cast(rows, _vp), len(group_rows), axis,
                                       int(colwise))


def _grouped_need(M, W, group_rows, axis):
    """Outputs of a grouped MXFP8 cast of quantised [rows][W] groups."""
    need = {}
    if axis & ROWWISE:
        need["q_row"] = ((M, W), U8)
        need["s_row"] = ((max(1, mx_grouped_scale_size(W, group_rows, axis, False)),), U8)
    if axis & COLWISE:
        need["q_col"] = ((M * W,), U8)
        need["s_col"] = ((max(1, mx_grouped_scale_size(W, group_rows, axis, True)),), U8)
    return need


def mx_quantize_grouped(x, group_rows, grad=None, axis=ROWWISE | COLWISE, fusion=FUSE_NONE,
                        out=None, workspace=None, stream=None):
    """Grouped MXFP8 cast of x[M][K] = len(group_rows) tensors stacked along
    rows.  Returns q_row [M][K], flat s_row / q_col / s_col holding the groups'
    outputs one after the other, and dbias [G][K] (None where not requested)."""
    x = _2d(x, "x")
    M, K = x.shape
    _group_total(group_rows, M)
    grad = _2d(grad, "grad") if (fusion & 0xF) in (FUSE_DGELU, FUSE_DSILU) else None
    _want_shape(grad, (M, K), "grad")
    G = len(group_rows)
    dev = x.device
    need = _grouped_need(M, K, group_rows, axis)
    if fusion & FUSE_DBIAS:
        need["dbias"] = ((G, K), F32)
    o = _outputs(out, need, dev)
    ws_bytes = 0
    if fusion & FUSE_DBIAS:
        workspace = _workspace(workspace,
                               mx_quantize_grouped_workspace_size(K, group_rows, axis, fusion), dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    _on_device(dev, grad, *o.values(), workspace if fusion & FUSE_DBIAS else None)
    rows = _rows_arg(group_rows)
    st = lib().mx_quantize_grouped(_ptr(x), _ptr(grad), K, ctypes.cast(rows, _vp), G, axis, fusion,
                                   _ptr(o.get("q_row")), _ptr(o.get("s_row")),
                                   _ptr(o.get("q_col")), _ptr(o.get("s_col")),
                                   _ptr(o.get("dbias")),
                                   _ptr(workspace) if fusion & FUSE_DBIAS else None, ws_bytes,
                                   _stream(dev, stream))
    _check(st, "mx_quantize_grouped")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col", "dbias")}


def mx_quantize_gated(x, act, axis=ROWWISE | COLWISE, out=None, stream=None):
    """Gated MXFP8 cast of x[M][2N] = [gate | linear] -> y[M][N] = act(gate)*linear."""
    x = _2d(x, "x")
    M, N2 = x.shape
    N = _half_width(N2, "mx_quantize_gated")
    dev = x.device
    o = _outputs(out, _mx_need(M, N, axis), dev)
    _on_device(dev, *o.values())
    st = lib().mx_quantize_gated(_ptr(x), M, N, axis, act, _ptr(o.get("q_row")),
                                 _ptr(o.get("s_row")), _ptr(o.get("q_col")),
                                 _ptr(o.get("s_col")), _stream(dev, stream))
    _check(st, "mx_quantize_gated")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col")}


def mx_quantize_dgated(grad, x, act, axis=ROWWISE | COLWISE, out=None, stream=None):
    """Gated backward MXFP8 cast: grad[M][N], x[M][2N] = [gate | linear] ->
    quantised dx[M][2N] = [d_gate | d_linear]."""
    grad = _2d(grad, "grad")
    x = _2d(x, "x")
    M, N2 = x.shape
    N = _half_width(N2, "mx_quantize_dgated")
    _want_shape(grad, (M, N), "grad")
    dev = x.device
    o = _outputs(out, _mx_need(M, N2, axis), dev)
    _on_device(dev, grad, *o.values())
    st = lib().mx_quantize_dgated(_ptr(grad), _ptr(x), M, N, axis, act, _ptr(o.get("q_row")),
                                  _ptr(o.get("s_row")), _ptr(o.get("q_col")),
                                  _ptr(o.get("s_col")), _stream(dev, stream))
    _check(st, "mx_quantize_dgated")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col")}


def mx_fused_values(x, grad=None, op=FUSE_GELU, out=None, stream=None):
    """The bf16 values the fused casts quantise (returned as int16 bits).
    Gated ops (OP_GATED | act) take x[M][2K] and give [M][K]; gated backward
    ops (OP_DGATED | act) take x[M][2K] and grad[M][K] and give [M][2K]."""
    x = _2d(x, "x")
    gated = bool(op & (OP_GATED | OP_DGATED))
    M, W = x.shape
    K = _half_width(W, "mx_fused_values") if gated else W
    dev = x.device
    shape = (M, 2 * K) if op & OP_DGATED else (M, K)
    g = _2d(grad, "grad") if (op in (FUSE_DGELU, FUSE_DSILU) or op & OP_DGATED) else None
    _want_shape(g, (M, K), "grad")
    y = _outputs({"y": out}, {"y": (shape, I16)}, dev)["y"]
    _on_device(dev, g, y)
    st = lib().mx_fused_values(_ptr(x), _ptr(g), M, K, op, _ptr(y), _stream(dev, stream))
    _check(st, "mx_fused_values")
    return y


def mx_absmax_bf16(x, out=None, stream=None):
    """Tensor absmax as a one-element float32 device tensor."""
    x = _bf16_bits(x)
    dev = x.device
    amax = _outputs({"amax": out}, {"amax": ((1,), F32)}, dev)["amax"]
    _on_device(dev, amax)
    st = lib().mx_absmax_bf16(_ptr(x), x.numel(), _ptr(amax), _stream(dev, stream))
    _check(st, "mx_absmax_bf16")
    return amax


def _nv_need(M, K, axis, n_sg):
    """NVFP4 outputs: codes [rows][ceil(cols/2)], scales [rows][ceil(cols/16)]."""
    need = {}
    if axis & ROWWISE:
        need["q_row"] = ((M, -(-K // 2)), U8)
        need["s_row"] = ((M, -(-K // 16)), U8)
    if axis & COLWISE:
        need["q_col"] = ((K, -(-M // 2)), U8)
        need["s_col"] = ((K, -(-M // 16)), U8)
    need["sg"] = ((n_sg,), F32)
    return need


def nvfp4_quantize_transpose(x, amax=None, axis=ROWWISE | COLWISE, out=None, stream=None,
                             two_d=False):
    """NVFP4 of x[M][K] and its transpose.  amax: one-element float32 device
    tensor (computed with mx_absmax_bf16 when None).  two_d: one scale per
    16 x 16 block.  Returns {q_row, s_row, q_col, s_col, sg}."""
    x = _2d(x, "x")
    M, K = x.shape
    dev = x.device
    o = _outputs(out, _nv_need(M, K, axis, 1), dev)
    if amax is not None:
        _f32_vec(amax, 1, "amax", dev)
    _on_device(dev, *o.values())
    if amax is None:
        amax = mx_absmax_bf16(x, stream=stream)
    fn = lib().nvfp4_quantize_transpose_2d if two_d else lib().nvfp4_quantize_transpose
    st = fn(_ptr(x), M, K, _ptr(amax), axis, _ptr(o.get("q_row")), _ptr(o.get("s_row")),
            _ptr(o.get("q_col")), _ptr(o.get("s_col")), _ptr(o["sg"]), _stream(dev, stream))
    _check(st, "nvfp4_quantize_transpose_2d" if two_d else "nvfp4_quantize_transpose")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col", "sg")}


def mx_absmax_bf16_grouped(x, group_rows, out=None, stream=None):
    """Per-group max |x| (fp32 [G]) of x[M][K] = len(group_rows) stacked tensors."""
    x = _2d(x, "x")
    M, K = x.shape
    _group_total(group_rows, M)
    G = len(group_rows)
    dev = x.device
    amax = _outputs({"amax": out}, {"amax": ((G,), F32)}, dev)["amax"]
    _on_device(dev, amax)
    rows = _rows_arg(group_rows)
    st = lib().mx_absmax_bf16_grouped(_ptr(x), K, ctypes.cast(rows, _vp), G, _ptr(amax),
                                      _stream(dev, stream))
    _check(st, "mx_absmax_bf16_grouped")
    return amax


def nvfp4_quantize_transpose_grouped(x, group_rows, amax, axis=ROWWISE | COLWISE, two_d=False,
                                     out=None, stream=None):
    """Grouped NVFP4 of x[M][K] = len(group_rows) stacked tensors, each with its
    own tensor amax (device fp32 [G]).  Returns q_row [M][ceil(K/2)], s_row
    [M][ceil(K/16)], flat q_col / s_col (the groups' transposes one after the
    other) and the groups' global scales sg [G]."""
    x = _2d(x, "x")
    M, K = x.shape
    _group_total(group_rows, M)
    G = len(group_rows)
    dev = x.device
    need = _nv_need(M, K, axis, G)
    if "q_col" in need:   # group g's [K][ceil(rows/2)] and [K][ceil(rows/16)], one after the other
        need["q_col"] = ((K * sum(-(-int(m) // 2) for m in group_rows),), U8)
        need["s_col"] = ((K * sum(-(-int(m) // 16) for m in group_rows),), U8)
    o = _outputs(out, need, dev)
    _f32_vec(amax, G, "amax", dev)
    _on_device(dev, *o.values())
    rows = _rows_arg(group_rows)
    st = lib().nvfp4_quantize_transpose_grouped(_ptr(x), K, ctypes.cast(rows, _vp), G, _ptr(amax),
                                                int(two_d), axis, _ptr(o.get("q_row")),
                                                _ptr(o.get("s_row")), _ptr(o.get("q_col")),
                                                _ptr(o.get("s_col")), _ptr(o["sg"]),
                                                _stream(dev, stream))
    _check(st, "nvfp4_quantize_transpose_grouped")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col", "sg")}


def mx_quantize_gated_grouped(x, group_rows, act, grad=None, axis=ROWWISE | COLWISE, out=None,
                              stream=None):
    """Grouped gated MXFP8 cast of x[M][2N] = [gate | linear] stacked by group
    (with grad [M][N]: the gated backward).  q_row [M][W] (W = N, or 2N
    backward) and flat s_row / q_col / s_col, the groups one after the other."""
    x = _2d(x, "x")
    M, N2 = x.shape
    N = _half_width(N2, "mx_quantize_gated_grouped")
    _group_total(group_rows, M)
    if grad is not None:
        grad = _2d(grad, "grad")
        _want_shape(grad, (M, N), "grad")
    W = N2 if grad is not None else N
    G = len(group_rows)
    dev = x.device
    o = _outputs(out, _grouped_need(M, W, group_rows, axis), dev)
    _on_device(dev, grad, *o.values())
    rows = _rows_arg(group_rows)
    ptrs = (_ptr(o.get("q_row")), _ptr(o.get("s_row")), _ptr(o.get("q_col")), _ptr(o.get("s_col")))
    if grad is None:
        st = lib().mx_quantize_gated_grouped(_ptr(x), N, ctypes.cast(rows, _vp), G, axis, act,
                                             *ptrs, _stream(dev, stream))
    else:
        st = lib().mx_quantize_dgated_grouped(_ptr(grad), _ptr(x), N, ctypes.cast(rows, _vp), G,
                                              axis, act, *ptrs, _stream(dev, stream))
    _check(st, "mx_quantize_gated_grouped")
    return {k: o.get(k) for k in ("q_row", "s_row", "q_col", "s_col")}


# ---- products on quantised operands -------------------------------------------

BF16 = torch.bfloat16


def _codes(t, name):
    """An operand's codes or scales: a contiguous uint8 tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype != U8:
        raise TypeError(f"{name} must be a uint8 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _want_bytes(t, n, name):
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} bytes, got {t.numel()}")


def _product_out(out, shape, flags, dev, stream):
    """The output tensor: bf16 (int16 / uint16 bits accepted in `out`) or, with
    OUT_F32, float32; ACCUMULATE needs the caller's."""
    dtype = F32 if flags & OUT_F32 else BF16
    if out is None:
        if flags & ACCUMULATE:
            raise ValueError("ACCUMULATE adds to `out`: it must be passed")
        return _empty(shape, dtype, dev, stream)
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a tensor")
    ok = out.dtype == dtype or (dtype == BF16 and out.dtype in (I16, torch.uint16))
    n = 1
    for d in shape:
        n *= d
    if not ok or out.numel() != n or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"out must be a contiguous {dtype} tensor of {n} elements on {dev}; got "
                         f"{out.dtype}, {out.numel()} elements on {out.device}")
    return out


def _empty(shape, dtype, dev, stream):
    """Device memory for work on `stream`: taken from that stream's pool, so that
    no other stream's pending work still uses it."""
    if stream is None or dev.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _group_rows(group_rows, M=None):
    """The group sizes as ints, checked as _group_total does."""
    rows = [int(r) for r in group_rows]
    if rows and min(rows) < 0 or M is not None and sum(rows) != M:
        _group_total(rows, M)
    return rows


def _group_scale_bytes(rows, cols, flags):
    """Bytes of the scales of operands [r][cols], r in rows, one after the other."""
    nb = -(-cols // 32)
    if flags & SCALE_TILED:
        return sum((r + 31) // 32 for r in rows) * -(-nb // 8) * 256
    return sum(rows) * nb


def _group_col_scale_bytes(rows, cols, flags):
    """The same of their transposed operands [cols][r]."""
    if flags & SCALE_TILED:
        return -(-cols // 32) * sum((r + 255) // 256 for r in rows) * 256
    return cols * sum((r + 31) // 32 for r in rows)


def _scale_bytes(rows, cols, flags):
    """Bytes of one operand's scales (none for an operand without elements)."""
    nb = -(-cols // 32)
    if flags & SCALE_TILED:
        return -(-rows // 32) * -(-nb // 8) * 256
    return rows * nb


def _current_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _current_device():
    return torch._C._cuda_getDevice()


def _launch(where, dev, stream, fn, *args):
    """Calls fn on the tensors' device (made current for the call) and stream.
    (The current stream's handle alone: making a torch.cuda.Stream of it takes 2
    of the 10 microseconds of a call.)"""
    handle = _current_stream(dev.index) if stream is None else stream.cuda_stream
    if dev.index == _current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        _check(st, where)


def _product_ws(workspace, need, dev, stream):
    """The products' workspace: (tensor to keep, pointer, bytes)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _empty((need,), U8, dev, stream)
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() \
            or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def mx_matmul_workspace_size(M: int, N: int, K: int, flags: int = 0) -> int:
    return lib().mx_matmul_workspace_size(M, N, K, flags)


def mx_matmul_grouped_workspace_size(N: int, K: int, group_rows, flags: int = 0) -> int:
    rows = _rows_arg(group_rows)
    return lib().mx_matmul_grouped_workspace_size(N, K, ctypes.addressof(rows), len(group_rows), flags)


def mx_matmul_wgrad_grouped_workspace_size(N: int, K: int, group_rows, flags: int = 0) -> int:
    rows = _rows_arg(group_rows)
    return lib().mx_matmul_wgrad_grouped_workspace_size(N, K, ctypes.addressof(rows),
                                                        len(group_rows), flags)


def mx_matmul(qa, sa, qb, sb, flags=0, out=None, workspace=None, stream=None):
    """y[M][N] = A B^T of MXFP8 operands quantised along K: codes qa [M][K],
    qb [N][K] and their scales sa, sb as the casts return them (compact, or in
    the tile layout with SCALE_TILED).  bf16, or float32 with OUT_F32; `out`
    may hold the output (with ACCUMULATE it is added to) and `workspace` the
    device scratch (mx_matmul_workspace_size bytes)."""
    for t, name in ((qa, "qa"), (sa, "sa"), (qb, "qb"), (sb, "sb")):
        _codes(t, name)
    if qa.dim() != 2 or qb.dim() != 2 or qa.shape[1] != qb.shape[1]:
        raise ValueError(f"qa [M][K] and qb [N][K] must be 2-D with one K, got "
                         f"{tuple(qa.shape)} and {tuple(qb.shape)}")
    (M, K), N, dev = qa.shape, qb.shape[0], qa.device
    _want_bytes(sa, _scale_bytes(M, K, flags), "sa")
    _want_bytes(sb, _scale_bytes(N, K, flags), "sb")
    y = _product_out(out, (M, N), flags, dev, stream)
    _on_device(dev, sa, qb, sb)
    L = lib()
    ws, wp, wn = _product_ws(workspace, L.mx_matmul_workspace_size(M, N, K, flags), dev, stream)
    _launch("mx_matmul", dev, stream, L.mx_matmul, qa.data_ptr(), sa.data_ptr(), qb.data_ptr(),
            sb.data_ptr(), M, N, K, flags, y.data_ptr(), wp, wn)
    return y


def mx_matmul_grouped(qa, sa, qb, sb, group_rows, flags=0, out=None, workspace=None, stream=None):
    """y[M][N]: each group's rows of A (codes qa [M][K], stacked as for
    mx_quantize_grouped, the groups' scales one after the other) by the group's
    own B_g [N][K] (codes qb and scales sb of the G matrices one after the
    other, any shape)."""
    for t, name in ((qa, "qa"), (sa, "sa"), (qb, "qb"), (sb, "sb")):
        _codes(t, name)
    if qa.dim() != 2:
        raise ValueError(f"qa must be 2-D, got shape {tuple(qa.shape)}")
    (M, K), G, dev = qa.shape, len(group_rows), qa.device
    rows = _group_rows(group_rows, M)
    if G == 0 or K == 0 or qb.numel() % (G * K):
        raise ValueError(f"qb must hold {G} matrices with rows of {K}, got {qb.numel()} bytes")
    N = qb.numel() // (G * K)
    _want_bytes(sa, _group_scale_bytes(rows, K, flags), "sa")
    _want_bytes(sb, G * _scale_bytes(N, K, flags), "sb")
    y = _product_out(out, (M, N), flags, dev, stream)
    _on_device(dev, sa, qb, sb)
    L, table = lib(), (ctypes.c_int64 * G)(*rows)
    rp = ctypes.addressof(table)
    ws, wp, wn = _product_ws(workspace, L.mx_matmul_grouped_workspace_size(N, K, rp, G, flags), dev,
                             stream)
    _launch("mx_matmul_grouped", dev, stream, L.mx_matmul_grouped, qa.data_ptr(), sa.data_ptr(),
            qb.data_ptr(), sb.data_ptr(), N, K, rp, G, flags, y.data_ptr(), wp, wn)
    return y


def mx_matmul_wgrad_grouped(qa, sa, qb, sb, group_rows, flags=0, out=None, workspace=None,
                            stream=None):
    """dW[G][N][K]: each group's sum over its rows m of dY[m][n] X[m][k], from
    the transposed outputs (q_col, s_col) of the grouped casts of dY [M][N]
    (qa, sa) and X [M][K] (qb, sb).  An empty group's gradient is 0 (with
    ACCUMULATE: unchanged)."""
    for t, name in ((qa, "qa"), (sa, "sa"), (qb, "qb"), (sb, "sb")):
        _codes(t, name)
    G, dev = len(group_rows), qa.device
    rows = _group_rows(group_rows)
    M = sum(rows)
    if M == 0 or qa.numel() % M or qb.numel() % M:
        raise ValueError(f"qa and qb must hold whole columns of {M} rows, got {qa.numel()} and "
                         f"{qb.numel()} bytes")
    N, K = qa.numel() // M, qb.numel() // M
    _want_bytes(sa, _group_col_scale_bytes(rows, N, flags), "sa")
    _want_bytes(sb, _group_col_scale_bytes(rows, K, flags), "sb")
    y = _product_out(out, (G, N, K), flags, dev, stream)
    _on_device(dev, sa, qb, sb)
    L, table = lib(), (ctypes.c_int64 * G)(*rows)
    rp = ctypes.addressof(table)
    ws, wp, wn = _product_ws(workspace, L.mx_matmul_wgrad_grouped_workspace_size(N, K, rp, G, flags),
                             dev, stream)
    _launch("mx_matmul_wgrad_grouped", dev, stream, L.mx_matmul_wgrad_grouped, qa.data_ptr(),
            sa.data_ptr(), qb.data_ptr(), sb.data_ptr(), N, K, rp, G, flags, y.data_ptr(), wp, wn)
    return y


def _nv_weights(x, qw, sw, sg, G):
    """Sizes of x [T][K] and G NVFP4 matrices [N][K] (codes [G * N][ceil(K/2)])."""
    x = _2d(x, "x")
    T, K = x.shape
    pitch, nb = -(-K // 2), -(-K // 16)
    _codes(qw, "qw")
    _codes(sw, "sw")
    if K == 0 or G == 0 or qw.numel() % (G * pitch):
        raise ValueError(f"qw must hold {G} matrices with rows of {pitch} bytes, got {qw.numel()}")
    N = qw.numel() // (G * pitch)
    _want_bytes(sw, G * N * nb, "sw")
    _f32_vec(sg, G, "sg", x.device)
    return T, N, K


def nvfp4_matvec(x, qw, sw, sg, flags=0, out=None, stream=None):
    """y[T][N] = x W^T: x bf16 [T][K], W [N][K] as nvfp4_quantize_transpose
    returns it (q_row, s_row, sg).  bf16, or float32 with OUT_F32."""
    T, N, K = _nv_weights(x, qw, sw, sg, 1)
    dev = x.device
    y = _product_out(out, (T, N), flags, dev, stream)
    _on_device(dev, qw, sw)
    _launch("nvfp4_matvec", dev, stream, lib().nvfp4_matvec, x.data_ptr(), T, qw.data_ptr(),
            sw.data_ptr(), sg.data_ptr(), N, K, flags, y.data_ptr())
    return y


def nvfp4_matvec_experts(x, experts, qw, sw, sg, flags=0, out=None, stream=None):
    """y[T][top][N]: y[t][j] = x[t] W_e^T with e = experts[t][j] (int32 [T][top])
    among the G = len(sg) stacked matrices qw [G * N][ceil(K/2)], sw; a row of
    zeros for an e outside 0 .. G - 1."""
    if not isinstance(sg, torch.Tensor) or not isinstance(experts, torch.Tensor):
        raise TypeError("sg and experts must be tensors")
    G = sg.numel()
    T, N, K = _nv_weights(x, qw, sw, sg, G)
    dev = x.device
    if experts.dtype != torch.int32 or experts.dim() != 2 or experts.shape[0] != T \
            or not experts.is_contiguous():
        raise ValueError(f"experts must be a contiguous int32 tensor [{T}][top], got "
                         f"{experts.dtype} {tuple(experts.shape)}")
    top = experts.shape[1]
    y = _product_out(out, (T, top, N), flags, dev, stream)
    _on_device(dev, experts, qw, sw)
    _launch("nvfp4_matvec_experts", dev, stream, lib().nvfp4_matvec_experts, x.data_ptr(),
            experts.data_ptr(), T, top, qw.data_ptr(), sw.data_ptr(), sg.data_ptr(), G, N, K, flags,
            y.data_ptr())
    return y


# ---- the norm before a product, the router, and the rows' way to the experts ----

I32 = torch.int32


_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)
_F32, _U8, _I32 = (F32,), (U8,), (I32,)


def _want(t, shape, dtypes, name, dev):
    """The address of an input, a contiguous tensor of this shape and one of these
    types on dev (None for None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous tensor {tuple(shape)} on {dev}; got "
                         f"{tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _new(like, out, stream):
    """A function of (name, shape, dtype) that gives outputs on the device of `like`:
    out's tensor of that name, of as many elements, or a new one (of the pool of the
    stream that works on it)."""
    if out is None and stream is None:
        empty = like.new_empty
        return lambda name, shape, dtype: empty(shape, dtype=dtype)
    dev = like.device

    def take(name, shape, dtype):
        t = None if out is None else out.get(name)
        if t is None:
            return _empty(shape, dtype, dev, stream)
        n = 1
        for d in shape:
            n *= d
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"out[{name!r}] must be a tensor")
        ok = t.dtype == dtype or (dtype == BF16 and t.dtype in _BF16_BITS)
        if not ok or t.numel() != n or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"out[{name!r}] must be a contiguous {dtype} tensor of {n} elements on "
                             f"{dev}; got {t.dtype}, {t.numel()} elements on {t.device}"
                             f"{'' if t.is_contiguous() else ', not contiguous'}")
        return t

    return take


def _at(t):
    return None if t is None else t.data_ptr()


def _gpu(dev):
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a ROCm (cuda) device, got {dev}")


def _scales_of(rows, cols, axis):
    """Shape of one direction's scales, as _scale_shape gives it."""
    if axis & SCALE_TILED:
        return (_scale_bytes(rows, cols, axis),)
    return (rows, -(-cols // 32))


def mx_rmsnorm_workspace_size(M: int, axis: int) -> int:
    return lib().mx_rmsnorm_workspace_size(M, axis)


def mx_rmsnorm(x, weight=None, residual=None, eps=1e-6, axis=0, want_y=None, checkpoint=False,
               out=None, workspace=None, stream=None):
    """h = x + residual (x itself without), y = h rstd weight with rstd =
    (mean h^2 + eps)^(-1/2) of each row, for bf16 x [M][K], and the MXFP8 casts
    of y that `axis` asks for (0: none; flags as for mx_quantize).  Returns {h, y,
    rstd, q_row, s_row, q_col, s_col, q_h, s_h}, None where not requested: y with
    want_y (default: without casts), q_h and s_h, an 8-bit copy of h for
    mx_rmsnorm_backward, with `checkpoint`.  Without a residual h is x."""
    x = _2d(x, "x")
    shape, dev = x.shape, x.device
    M, K = shape
    rp = _want(residual, shape, _BF16_BITS, "residual", dev)
    wp = _want(weight, (K,), _BF16_BITS, "weight", dev)
    h = y = q_row = s_row = q_col = s_col = q_h = s_h = ws = wp_ = None
    wn = 0
    new = _new(x, out, stream)
    if residual is not None:
        h = new("h", shape, BF16)
    if want_y or (want_y is None and not axis):
        y = new("y", shape, BF16)
    rstd = new("rstd", (M,), F32)
    if axis & ROWWISE:
        q_row, s_row = new("q_row", shape, U8), new("s_row", _scales_of(M, K, axis), U8)
    if axis & COLWISE:
        q_col, s_col = new("q_col", (K, M), U8), new("s_col", _scales_of(K, M, axis), U8)
        if workspace is None:
            ws, wn = new("workspace", (2 * M,), F32), 8 * M
            wp_ = ws.data_ptr()
        else:
            ws, wp_, wn = _product_ws(workspace, 8 * M, dev, stream)
    if checkpoint:
        q_h, s_h = new("q_h", shape, U8), new("s_h", (M, -(-K // 32)), U8)
    if dev.index is None:
        _gpu(dev)
    _launch("mx_rmsnorm", dev, stream, lib().mx_rmsnorm, x.data_ptr(), rp, wp, M, K, eps, axis, _at(h),
            _at(y), _at(q_row), _at(s_row), _at(q_col), _at(s_col), _at(q_h), _at(s_h), rstd.data_ptr(),
            wp_, wn)
    return {"h": x if h is None else h, "y": y, "rstd": rstd, "q_row": q_row, "s_row": s_row,
            "q_col": q_col, "s_col": s_col, "q_h": q_h, "s_h": s_h}


def mx_rmsnorm_backward_workspace_size(M: int, K: int) -> int:
    return lib().mx_rmsnorm_backward_workspace_size(M, K)


def mx_rmsnorm_backward(dy, rstd, weight=None, h=None, q_h=None, s_h=None, dres=None,
                        want_dweight=True, out=None, workspace=None, stream=None):
    """Gradients of mx_rmsnorm from dy, the gradient of y, the forward's rstd, and
    its h or the 8-bit copy q_h, s_h.  Returns {dh, dweight}: dh bf16 [M][K], the
    gradient of x and of the residual, with dres (that of h itself, from the
    residual stream) added; dweight float32 [K] (None without want_dweight)."""
    dy = _2d(dy, "dy")
    (M, K), dev = dy.shape, dy.device
    if (h is None) == (q_h is None) or (q_h is None) != (s_h is None):
        raise ValueError("mx_rmsnorm_backward takes either h or q_h and s_h")
    rp = _want(rstd, (M,), _F32, "rstd", dev)
    hp = _want(h, dy.shape, _BF16_BITS, "h", dev)
    qp = _want(q_h, dy.shape, _U8, "q_h", dev)
    sp = _want(s_h, (M, -(-K // 32)), _U8, "s_h", dev)
    wp = _want(weight, (K,), _BF16_BITS, "weight", dev)
    dp = _want(dres, dy.shape, _BF16_BITS, "dres", dev)
    new = _new(dy, out, stream)
    o = dict(dh=new("dh", (M, K), BF16), dweight=None)
    ws, pp, pn = None, None, 0
    L = lib()
    if want_dweight:
        o["dweight"] = new("dweight", (K,), F32)
        ws, pp, pn = _product_ws(workspace, L.mx_rmsnorm_backward_workspace_size(M, K), dev, stream)
    if dev.index is None:
        _gpu(dev)
    _launch("mx_rmsnorm_backward", dev, stream, L.mx_rmsnorm_backward, dy.data_ptr(), hp, qp, sp, rp,
            wp, dp, M, K, o["dh"].data_ptr(), _at(o["dweight"]), pp, pn)
    return o


def _logits(t):
    if not isinstance(t, torch.Tensor) or t.dtype not in (BF16, F32):
        raise TypeError("logits must be a bfloat16 or float32 tensor")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"logits must be a contiguous 2-D tensor, got {tuple(t.shape)}")
    return _ROUTE_F32 if t.dtype == F32 else 0


def moe_route(logits, top, bias=None, flags=0, groups=1, top_groups=1, scale=1.0, want_scores=False,
              out=None, stream=None):
    """Each token's `top` experts from its logits [T][E] (bf16 or float32), by
    softmax scores (sigmoid with ROUTE_SIGMOID) plus bias (float32 [E]), within the
    best top_groups of `groups` groups.  Returns {experts (int32 [T][top], -1:
    none), weights (float32 [T][top]: the scores without the bias, divided by their
    sum with ROUTE_RENORM, times scale), scores (float32 [T][E] with want_scores)}."""
    f32 = _logits(logits)
    (T, E), dev = logits.shape, logits.device
    bp = _want(bias, (E,), _F32, "bias", dev)
    new = _new(logits, out, stream)
    o = dict(experts=new("experts", (T, top), I32),
             weights=new("weights", (T, top), F32),
             scores=new("scores", (T, E), F32) if want_scores else None)
    if dev.index is None:
        _gpu(dev)
    _launch("moe_route", dev, stream, lib().moe_route, logits.data_ptr(), bp, T, E, top, groups,
            top_groups, scale, flags | f32, o["experts"].data_ptr(), o["weights"].data_ptr(),
            _at(o["scores"]))
    return o


def moe_route_backward(dweights, logits, experts, flags=0, scale=1.0, dscores=None, out=None,
                       stream=None):
    """The gradient of moe_route's logits (a tensor of their shape and type; `out`
    may hold it) from those of its weights and, with dscores, of its scores; flags
    and scale as in the forward."""
    f32 = _logits(logits)
    (T, E), dev = logits.shape, logits.device
    if not isinstance(experts, torch.Tensor) or experts.dim() != 2:
        raise ValueError("experts must be a tensor [T][top]")
    top = experts.shape[1]
    ep = _want(experts, (T, top), _I32, "experts", dev)
    wp = _want(dweights, (T, top), _F32, "dweights", dev)
    sp = _want(dscores, (T, E), _F32, "dscores", dev)
    o = _new(logits, None if out is None else {"out": out}, stream)("out", (T, E), logits.dtype)
    if dev.index is None:
        _gpu(dev)
    _launch("moe_route_backward", dev, stream, lib().moe_route_backward, logits.data_ptr(), ep, wp, sp,
            T, E, top, scale, flags | f32, o.data_ptr())
    return o


def moe_sort_rows(T: int, top: int, E: int, align: int = 1) -> int:
    return lib().moe_sort_rows(T, top, E, align)


def moe_sort_workspace_size(T: int, top: int, E: int) -> int:
    return lib().moe_sort_workspace_size(T, top, E)


def _slots_2d(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype != I32 or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [T][top]")
    return t


def moe_sort(experts, E, align=1, rows=None, out=None, workspace=None, stream=None):
    """The order of the slots (token, choice) of experts int32 [T][top] by expert,
    each expert's rows from a multiple of `align` on.  Returns {counts int32 [E],
    pos int32 [T][top] (each slot's row or -1), slots int32 [rows] (each row's slot
    or -1)}; rows: by default moe_sort_rows(T, top, E, align), the most there can
    be.  group_rows[e] of the grouped casts and products is counts[e] rounded up to
    align."""
    T, top = _slots_2d(experts, "experts").shape
    dev, L = experts.device, lib()
    rows = L.moe_sort_rows(T, top, E, align) if rows is None else int(rows)
    new = _new(experts, out, stream)
    o = dict(counts=new("counts", (E,), I32),
             pos=new("pos", (T, top), I32),
             slots=new("slots", (rows,), I32))
    ws, wp, wn = _product_ws(workspace, L.moe_sort_workspace_size(T, top, E), dev, stream)
    if dev.index is None:
        _gpu(dev)
    _launch("moe_sort", dev, stream, L.moe_sort, experts.data_ptr(), T, top, E, align, rows,
            o["counts"].data_ptr(), o["pos"].data_ptr(), o["slots"].data_ptr(), wp, wn)
    return o


def moe_gather(x, slots, top, out=None, stream=None):
    """Row r of the result [rows][...] is row slots[r] // top of x [T][...] (any
    type), or zeros where slots[r] names no slot."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be a contiguous tensor [T][...]")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D tensor")
    dev, T, rows = x.device, x.shape[0], slots.shape[0]
    sp = _want(slots, (rows,), _I32, "slots", dev)
    o = _new(x, None if out is None else {"out": out}, stream)("out", (rows, *x.shape[1:]), x.dtype)
    width = x.element_size()
    for d in x.shape[1:]:
        width *= d
    if dev.index is None:
        _gpu(dev)
    _launch("moe_gather", dev, stream, lib().moe_gather, x.data_ptr(), T, top, sp, rows, width,
            o.data_ptr())
    return o


def _rows_and_slots(y, weights, pos):
    """(T, top, rows, K) of experts' rows y: [rows][K] with pos [T][top], or
    [T][top][K]."""
    y = _bf16_bits(y)
    if pos is None:
        if y.dim() != 3:
            raise ValueError(f"without pos y must be [T][top][K], got {tuple(y.shape)}")
        T, top, K = y.shape
        rows = T * top
    else:
        T, top = _slots_2d(pos, "pos").shape
        if y.dim() != 2:
            raise ValueError(f"y must be [rows][K], got {tuple(y.shape)}")
        rows, K = y.shape
    dev = y.device
    pp = _want(pos, (T, top), _I32, "pos", dev)
    wp = _want(weights, (T, top), _F32, "weights", dev)
    return T, top, rows, K, pp, wp


def moe_combine(y, weights=None, pos=None, out=None, stream=None):
    """out[t] = sum_j weights[t][j] y[pos[t][j]] (bf16 [T][K]) of the experts' rows
    y bf16 [rows][K]; a pos that names no row adds nothing.  Without pos y is
    [T][top][K], as nvfp4_matvec_experts returns it; without weights they are 1."""
    T, top, rows, K, pp, wp = _rows_and_slots(y, weights, pos)
    dev = y.device
    o = _new(y, None if out is None else {"out": out}, stream)("out", (T, K), BF16)
    if dev.index is None:
        _gpu(dev)
    _launch("moe_combine", dev, stream, lib().moe_combine, y.data_ptr(), rows, K, pp, wp, T, top,
            o.data_ptr())
    return o


def moe_combine_backward(dout, y, weights=None, pos=None, slots=None, want_dweights=True, out=None,
                         stream=None):
    """Gradients of moe_combine from that of its output, dout bf16 [T][K]: {dy (of
    y's shape, zeros in rows without a slot), dweights (float32 [T][top])}.  With
    pos, slots as moe_sort returned it: a row whose slot's pos is another row is not
    written."""
    T, top, rows, K, pp, wp = _rows_and_slots(y, weights, pos)
    dev = y.device
    if (pos is None) != (slots is None):
        raise ValueError("pos and slots go together")
    gp = _want(dout, (T, K), _BF16_BITS, "dout", dev)
    sp = _want(slots, (rows,), _I32, "slots", dev)
    new = _new(y, out, stream)
    o = dict(dy=new("dy", tuple(y.shape), BF16),
             dweights=new("dweights", (T, top), F32) if want_dweights else None)
    if dev.index is None:
        _gpu(dev)
    _launch("moe_combine_backward", dev, stream, lib().moe_combine_backward, gp, y.data_ptr(), rows, K,
            pp, sp, wp, T, top, o["dy"].data_ptr(), _at(o["dweights"]))
    return o
