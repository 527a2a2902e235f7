"""Python binding of libmoe.so, the MI355X 4-bit group-affine MoE layer.

Argument marshalling only: every function forwards device pointers (taken
from torch tensors with ``.data_ptr()``) and the current HIP stream to the C
ABI declared in include/moe.h, and raises MoEError on a non-OK status.  The
calls beside the layer (microscaled 4-bit, balance loss, routing from scores,
combination, adapters) check their tensors' types, sizes and device as well.
All computation happens in the library's HIP kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARGUMENT", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_HIP", 5: "MOE_ERR_DEVICE_UNSUPPORTED"}

# Kernel ids of moe_profile_read.
(K_LOGITS, K_TOPK, K_META, K_GATEUP_GEMM, K_DOWN_GEMM, K_GATEUP_GEMV, K_DOWN_GEMV, K_COMBINE, K_DEQUANT,
 K_PROBE_READ, K_PROBE_MFMA, K_MX4_QUANTIZE, K_MX4_DEQUANTIZE,
 K_MX4_EXPERTS, K_BALANCE, K_BALANCE_GRAD, K_SELECT, K_SELECT_GRAD, K_SORT, K_COMBINE_ROWS, K_COMBINE_GRAD,
 K_ADAPTERS, K_ADAPTERS_GRAD) = range(23)
KERNEL_NAMES = {K_LOGITS: "k_screen|k_logits_small", K_TOPK: "k_route_exact", K_META: "k_meta|k_topk_meta",
                K_GATEUP_GEMM: "k_gateup_gemm", K_DOWN_GEMM: "k_down_gemm",
                K_GATEUP_GEMV: "k_gemv_experts", K_DOWN_GEMV: "k_gemv_reduce", K_COMBINE: "k_combine",
                K_DEQUANT: "k_dequant_active", K_PROBE_READ: "k_stream_read", K_PROBE_MFMA: "k_mfma_rate",
                K_MX4_QUANTIZE: "k_mx4_quantize", K_MX4_DEQUANTIZE: "k_mx4_dequantize",
                K_MX4_EXPERTS: "k_mx4_few|k_mx4_grid",
                K_BALANCE: "k_balance_rows|k_balance_sum", K_BALANCE_GRAD: "k_balance_grad",
                K_SELECT: "k_select|k_sort_scan|k_sort_place", K_SELECT_GRAD: "k_select_grad",
                K_SORT: "k_sort_count|k_sort_scan|k_sort_place", K_COMBINE_ROWS: "k_combine_rows",
                K_COMBINE_GRAD: "k_combine_grad", K_ADAPTERS: "k_adapters_rows",
                K_ADAPTERS_GRAD: "k_adapters_rows|k_adapters_sums"}

# Element types of the calls beside the layer.
MOE_F32, MOE_BF16, MOE_MX4 = range(3)

# Scores of moe_select_forward.
MOE_SOFTMAX, MOE_SIGMOID = range(2)


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class LayerDesc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("hidden", "n_experts", "top_k", "inter", "shared_inter",
                                         "group_size", "gemv_max_rows", "max_chunk", "tile_rows",
                                         "host_sync_routing", "dequant_pass", "batch_invariant")]


class Mx4Desc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_experts", "n", "k", "x_type", "y_type", "swiglu")]


class SelectDesc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_experts", "top_k", "scores", "n_groups", "top_groups", "group_best",
                                         "renormalise")] + [("scale", C.c_float)]


class AdapterDesc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_adapters", "rank", "n_in", "n_out", "y_type")]


class QMatrix(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("biases", C.c_void_p)]


class Routing(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("topk_ids", "topk_weights", "expert_counts",
                                          "expert_offsets", "sorted_assign", "tile_map", "n_tiles")]


_lib = None


def lib():
    """Load libmoe.so (built by bit_quantized_moe_router_amd/build.py); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python bit_quantized_moe_router_amd/build.py`")
        # torch carries its own HIP runtime (same soname as ROCm's).  Loading it
        # first makes libmoe.so bind to that one; loaded the other way round the
        # process would hold two HIP runtimes, and the second to open the GPU
        # finds no device.
        import torch  # noqa: F401
        L = C.CDLL(LIB_PATH)
        P, vp, i32, sz = C.POINTER, C.c_void_p, C.c_int32, C.c_size_t
        D = P(LayerDesc)
        L.moe_packed_bytes.argtypes = [D, P(sz)]
        L.moe_workspace_bytes.argtypes = [D, i32, P(sz)]
        L.moe_max_tiles.argtypes = [D, i32, P(i32)]
        L.moe_pack_weights.argtypes = [D, QMatrix, QMatrix, QMatrix, QMatrix, QMatrix, QMatrix, vp, sz, vp]
        L.moe_route.argtypes = [D, vp, i32, vp, vp, P(Routing), vp, sz, vp]
        L.moe_forward_prefill.argtypes = [D, vp, vp, vp, vp, i32, vp, vp, sz, vp]
        L.moe_forward_decode.argtypes = [D, vp, vp, vp, vp, i32, vp, vp, sz, vp]
        L.moe_forward_decode_static.argtypes = [D, vp, vp, vp, vp, i32, vp, vp]
        L.moe_default_gemv_max_rows.argtypes = []
        L.moe_default_gemv_max_rows.restype = i32
        L.moe_status_str.argtypes = [C.c_int]
        L.moe_status_str.restype = C.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = C.c_char_p
        L.moe_mx4_experts_kernel.argtypes = []
        L.moe_mx4_experts_kernel.restype = C.c_char_p
        L.moe_probe_stream_read.argtypes = [vp, sz, vp, i32, vp]
        L.moe_probe_mfma_rate.argtypes = [i32, i32, vp, vp, vp]
        L.moe_profile_enable.argtypes = [i32]
        L.moe_profile_reset.argtypes = []
        L.moe_profile_read.argtypes = [i32, P(C.c_double), P(i32)]
        i64 = C.c_int64
        L.moe_mx4_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
        L.moe_mx4_dequantize.argtypes = [vp, vp, i64, i64, vp, i32, i64, vp]
        L.moe_mx4_experts.argtypes = [P(Mx4Desc), vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, vp, vp, vp, i32, vp]
        f32 = C.c_float
        L.moe_balance_loss_workspace_bytes.argtypes = [i32, i32, P(sz)]
        L.moe_balance_loss_forward.argtypes = [vp, i32, i32, i32, vp, i32, vp, f32, f32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_balance_loss_backward.argtypes = [vp, i32, i32, i32, i32, vp, f32, f32, vp, vp, vp, vp, vp]
        S, A = P(SelectDesc), P(AdapterDesc)
        L.moe_select_workspace_bytes.argtypes = [i32, i32, i32, P(sz)]
        L.moe_select_forward.argtypes = [S, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_select_backward.argtypes = [S, vp, i32, i32, vp, vp, vp, vp, vp, vp]
        L.moe_sort_workspace_bytes.argtypes = [i32, i32, P(sz)]
        L.moe_sort_assignments.argtypes = [vp, i32, i32, vp, vp, vp, vp, sz, vp]
        L.moe_combine_forward.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, i32, vp]
        L.moe_combine_backward.argtypes = [vp, i32, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_adapters_forward.argtypes = [A, vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, vp, vp, i32, vp, vp]
        L.moe_adapters_workspace_bytes.argtypes = [A, i32, P(sz)]
        L.moe_adapters_backward.argtypes = [A, vp, vp, vp, vp, i32, vp, vp, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp,
                                            sz, vp]
        for name in ("moe_select_workspace_bytes", "moe_select_forward", "moe_select_backward", "moe_sort_workspace_bytes",
                     "moe_sort_assignments", "moe_combine_forward", "moe_combine_backward", "moe_adapters_forward",
                     "moe_adapters_workspace_bytes", "moe_adapters_backward", "moe_balance_loss_workspace_bytes", "moe_balance_loss_forward", "moe_balance_loss_backward",
                     "moe_mx4_experts", "moe_mx4_quantize", "moe_mx4_dequantize", "moe_packed_bytes", "moe_workspace_bytes", "moe_max_tiles", "moe_pack_weights",
                     "moe_route", "moe_forward_prefill", "moe_forward_decode", "moe_forward_decode_static",
                     "moe_probe_stream_read", "moe_probe_mfma_rate", "moe_profile_enable",
                     "moe_profile_reset", "moe_profile_read"):
            getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise MoEError(status, lib().moe_last_error().decode())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream().cuda_stream


# The calls from here to make_desc check their tensors' types, sizes and device,
# so that a pointer never stands for less memory than the kernel takes it for,
# and put their work on the tensors' device.  A decode step's call is bound by
# this code, so the checks look at little and make no objects.

def _bad(message, status=1):
    raise MoEError(status, message)


def _int32(value, name):
    """value, for an int32_t of the library, of which ctypes would pass the low 32 bits alone."""
    return value if -0x80000000 <= value <= 0x7FFFFFFF else _bad(f"{name} does not fit 32 bits (got {value})", 2)


def _value_type(t, name):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return MOE_BF16
    return MOE_F32 if t.dtype is torch.float32 else _bad(f"{name} must be bfloat16 or float32 (got {t.dtype})")


def _arg(t, name, dtype, numel, dev, width=None):
    """The address of a contiguous tensor of this type, size and device index; a matrix has rows of `width`
    elements (whatever stands before them), or is flat."""
    if (t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or not t.is_contiguous()
            or width is not None and t.dim() > 1 and t.shape[-1] != width):
        rows = "" if width is None else f" in rows of {width}"
        _bad(f"{name} must be a contiguous {dtype} tensor of {numel} elements{rows} on the call's device "
             f"(got {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, {t.device})")
    return t.data_ptr()


def _on_device(dev, stream, call, *args):
    """call(*args, stream) with device `dev` current; stream None is that device's current one."""
    torch = _torch()
    if dev < 0:
        _bad("the tensors must be on a GPU")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        status = call(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = call(*args, stream)
    if status != 0:
        _check(status)


def _mx4_rows(v, name, codes, scales):
    torch = _torch()
    if v.dim() != 2:
        _bad(f"{name} must be 2-D (got {tuple(v.shape)})")
    rows, cols = v.shape
    ld, one = v.stride()
    if one != 1 and cols > 1 or ld < cols and rows > 1:
        _bad(f"{name} must have rows of consecutive values (got {tuple(v.shape)}, strides {v.stride()})")
    if cols == 0 or cols % 32:
        _bad(f"cols must be a positive multiple of 32 (got {cols})", 2)
    dev = v.get_device()
    return (_value_type(v, name), rows, cols, ld if rows > 1 else cols, dev,
            _arg(codes, "codes", torch.uint8, rows * cols // 2, dev, cols // 2),
            _arg(scales, "scales", torch.uint8, rows * cols // 32, dev, cols // 32))


def moe_mx4_quantize(x, codes, scales, stream=None):
    """x [rows, cols] float32 or bfloat16 -> codes [rows, cols/2], scales [rows, cols/32] (uint8)."""
    kind, rows, cols, ld, dev, c, s = _mx4_rows(x, "x", codes, scales)
    _on_device(dev, stream, lib().moe_mx4_quantize, x.data_ptr(), kind, rows, cols, ld, c, s)


def moe_mx4_dequantize(codes, scales, y, stream=None):
    """codes, scales as moe_mx4_quantize writes them -> y [rows, cols] float32 or bfloat16."""
    kind, rows, cols, ld, dev, c, s = _mx4_rows(y, "y", codes, scales)
    _on_device(dev, stream, lib().moe_mx4_dequantize, c, s, rows, cols, y.data_ptr(), kind, ld)


def make_mx4_desc(n_experts, n, k, x_type, y_type, swiglu=0) -> Mx4Desc:
    return Mx4Desc(_int32(n_experts, "n_experts"), _int32(n, "n"), _int32(k, "k"), x_type, y_type, swiglu)


def _rows(t, name, kind, cols, scales, dev):
    """(rows, address, scales' address) of a 2-D operand of type `kind` with `cols` values a row."""
    torch = _torch()
    if kind == MOE_MX4:
        dtype, width = torch.uint8, cols // 2
    else:
        dtype, width = torch.float32 if kind == MOE_F32 else torch.bfloat16, cols
    if t.dim() != 2 or t.shape[1] != width:
        _bad(f"{name} must be 2-D with {width} columns (got {tuple(t.shape)})")
    rows = _int32(t.shape[0], f"the number of {name}'s rows")
    p = _arg(t, name, dtype, rows * width, dev)
    if kind == MOE_MX4:
        if scales is None:
            _bad(f"{name}_scales is missing")
        return rows, p, _arg(scales, name + "_scales", torch.uint8, rows * (cols // 32), dev, cols // 32)
    if scales is not None:
        _bad(f"{name}_scales goes with a MOE_MX4 {name} only")
    return rows, p, None


def moe_mx4_experts(desc, w_codes, w_scales, x, x_scales, expert_offsets, rows, y, y_scales=None, src_rows=None,
                    src_div=1, dst_rows=None, row_scale=None, stream=None):
    """Position i of expert e's range gives y[dst_rows[i]] = row_scale * W_e x[src_rows[i] // src_div]."""
    torch = _torch()
    E, n, k, x_type, y_type = desc.n_experts, desc.n, desc.k, desc.x_type, desc.y_type
    if x_type not in (MOE_BF16, MOE_MX4) or y_type not in (MOE_F32, MOE_BF16, MOE_MX4):
        _bad(f"x_type must be MOE_BF16 or MOE_MX4, y_type one of the three types (got {x_type}, {y_type})")
    if k <= 0 or k % 32:
        _bad(f"k must be a positive multiple of 32 (got {k})", 2)
    dev, i32 = x.get_device(), torch.int32
    wc = _arg(w_codes, "w_codes", torch.uint8, E * n * (k // 2), dev, k // 2)
    ws = _arg(w_scales, "w_scales", torch.uint8, E * n * (k // 32), dev, k // 32)
    off = _arg(expert_offsets, "expert_offsets", i32, E + 1, dev)
    rows, src_div = _int32(rows, "rows"), _int32(src_div, "src_div")
    x_rows, xp, xs = _rows(x, "x", x_type, k, x_scales, dev)
    y_rows, yp, ys = _rows(y, "y", y_type, n // 2 if desc.swiglu else n, y_scales, dev)
    src = None if src_rows is None else _arg(src_rows, "src_rows", i32, rows, dev)
    dst = None if dst_rows is None else _arg(dst_rows, "dst_rows", i32, rows, dev)
    fac = None if row_scale is None else _arg(row_scale, "row_scale", torch.float32, y_rows, dev)
    _on_device(dev, stream, lib().moe_mx4_experts, C.byref(desc), wc, ws, xp, xs, x_rows, off, rows, src, src_div, dst,
               fac, yp, ys, y_rows)


def moe_mx4_experts_kernel() -> str:
    """The kernel that this thread's last moe_mx4_experts call took (moe.h lists them)."""
    return lib().moe_mx4_experts_kernel().decode()


def moe_balance_loss_workspace_bytes(T: int, n_experts: int) -> int:
    n = C.c_size_t()
    _check(lib().moe_balance_loss_workspace_bytes(_int32(T, "T"), _int32(n_experts, "n_experts"), C.byref(n)))
    return n.value


def _logits(logits, valid):
    """(T, E, type, device index, address, valid's address)."""
    torch = _torch()
    if logits.dim() != 2 or not logits.is_contiguous():
        _bad(f"logits must be 2-D and contiguous (got {tuple(logits.shape)}, strides {logits.stride()})")
    T, E = logits.shape
    _int32(T, "T"), _int32(E, "n_experts")
    dev = logits.get_device()
    v = None
    if valid is not None:
        v = _arg(valid, "valid", torch.bool if valid.dtype is torch.bool else torch.uint8, T, dev)
    return T, E, _value_type(logits, "logits"), dev, logits.data_ptr(), v


def moe_balance_loss_forward(logits, topk_ids, valid, balance_coef, z_coef, losses, counts, mean_prob, n_valid, ws,
                             stream=None):
    """logits [T, E], topk_ids [T, k] int32, valid [T] uint8/bool or None -> losses [3] (loss, balance, z),
    counts [E] int32, mean_prob [E], n_valid [1] int32."""
    torch = _torch()
    T, E, kind, dev, p, v = _logits(logits, valid)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        _bad(f"topk_ids must be [T, k] (got {tuple(topk_ids.shape)} for T = {T})")
    k, i32, f32 = _int32(topk_ids.shape[1], "top_k"), torch.int32, torch.float32
    _on_device(dev, stream, lib().moe_balance_loss_forward, p, kind, T, E, _arg(topk_ids, "topk_ids", i32, T * k, dev),
               k, v, balance_coef, z_coef, _arg(losses, "losses", f32, 3, dev), _arg(counts, "counts", i32, E, dev),
               _arg(mean_prob, "mean_prob", f32, E, dev), _arg(n_valid, "n_valid", i32, 1, dev),
               _arg(ws, "ws", torch.uint8, ws.numel(), dev), ws.numel())


def moe_balance_loss_backward(logits, top_k, valid, balance_coef, z_coef, counts, n_valid, grad_loss, dlogits,
                              stream=None):
    """Gradient of moe_balance_loss_forward's loss; grad_loss [1] float32 or None (1)."""
    torch = _torch()
    T, E, kind, dev, p, v = _logits(logits, valid)
    _on_device(dev, stream, lib().moe_balance_loss_backward, p, kind, T, E, _int32(top_k, "top_k"), v, balance_coef, z_coef,
               _arg(counts, "counts", torch.int32, E, dev), _arg(n_valid, "n_valid", torch.int32, 1, dev),
               None if grad_loss is None else _arg(grad_loss, "grad_loss", torch.float32, 1, dev),
               _arg(dlogits, "dlogits", logits.dtype, T * E, dev, E))


def _bytes(ws, dev):
    """(address, bytes) of a workspace, None for none."""
    return (None, 0) if ws is None else (_arg(ws, "ws", _torch().uint8, ws.numel(), dev), ws.numel())


def _matrix(t, name, rows, cols, dev=None):
    """(type, address) of a contiguous float32 or bfloat16 matrix of this shape, (None, None) of None."""
    if t is None:
        return None, None
    kind = _value_type(t, name)
    if t.shape != (rows, cols) or not t.is_contiguous() or t.get_device() != dev:
        _bad(f"{name} must be a contiguous [{rows}, {cols}] tensor on the call's device (got {tuple(t.shape)}, strides "
             f"{t.stride()}, {t.device})")
    return kind, t.data_ptr()


def _same_type(kind, of, names):
    if kind is not None and kind != of:
        _bad(f"{names} must have one type")


def make_select_desc(n_experts, top_k, scores=MOE_SOFTMAX, n_groups=1, top_groups=1, group_best=1, renormalise=1,
                     scale=1.0) -> SelectDesc:
    sizes = dict(n_experts=n_experts, top_k=top_k, scores=scores, n_groups=n_groups, top_groups=top_groups,
                 group_best=group_best, renormalise=renormalise)
    return SelectDesc(*(_int32(v, name) for name, v in sizes.items()), scale)


def moe_select_workspace_bytes(T: int, n_experts: int, top_k: int) -> int:
    n = C.c_size_t()
    _check(lib().moe_select_workspace_bytes(_int32(T, "T"), _int32(n_experts, "n_experts"), _int32(top_k, "top_k"),
                                            C.byref(n)))
    return n.value


def _select_logits(desc, logits):
    """(T, E, k, type, device index, address)."""
    if logits.dim() != 2 or logits.shape[1] != desc.n_experts or not logits.is_contiguous():
        _bad(f"logits must be a contiguous [T, {desc.n_experts}] tensor (got {tuple(logits.shape)}, strides "
             f"{logits.stride()})")
    return (_int32(logits.shape[0], "T"), desc.n_experts, desc.top_k, _value_type(logits, "logits"), logits.get_device(),
            logits.data_ptr())


def moe_select_forward(desc, logits, bias, valid, topk_ids, topk_weights, expert_counts=None, expert_offsets=None,
                       sorted_assign=None, ws=None, stream=None):
    """logits [T, E], bias [E] float32 or None, valid [T] uint8/bool or None -> topk_ids [T, k] int32, topk_weights [T, k],
    and, or all None, expert_counts [E], expert_offsets [E + 1], sorted_assign [T * k] int32."""
    torch = _torch()
    T, E, k, kind, dev, p = _select_logits(desc, logits)
    i32, f32 = torch.int32, torch.float32
    b = None if bias is None else _arg(bias, "bias", f32, E, dev)
    v = None if valid is None else _arg(valid, "valid", torch.bool if valid.dtype is torch.bool else torch.uint8, T, dev)
    order = (None, None, None)
    if expert_counts is not None or expert_offsets is not None or sorted_assign is not None:
        if expert_counts is None or expert_offsets is None or sorted_assign is None:
            _bad("expert_counts, expert_offsets and sorted_assign go together")
        order = (_arg(expert_counts, "expert_counts", i32, E, dev), _arg(expert_offsets, "expert_offsets", i32, E + 1, dev),
                 _arg(sorted_assign, "sorted_assign", i32, T * k, dev, k if sorted_assign.dim() > 1 else None))
    _on_device(dev, stream, lib().moe_select_forward, C.byref(desc), p, kind, T, b, v,
               _arg(topk_ids, "topk_ids", i32, T * k, dev, k), _arg(topk_weights, "topk_weights", f32, T * k, dev, k), *order,
               *_bytes(ws, dev))


def moe_select_backward(desc, logits, topk_ids, topk_weights, dweights, base, dlogits, stream=None):
    """dlogits = base (or zeros) + the gradient of moe_select_forward's weights for dweights [T, k]."""
    torch = _torch()
    T, E, k, kind, dev, p = _select_logits(desc, logits)
    f32 = torch.float32
    base_kind, bp = _matrix(base, "base", T, E, dev)
    d_kind, dp = _matrix(dlogits, "dlogits", T, E, dev)
    _same_type(base_kind, kind, "base and logits")
    _same_type(d_kind, kind, "dlogits and logits")
    _on_device(dev, stream, lib().moe_select_backward, C.byref(desc), p, kind, T,
               _arg(topk_ids, "topk_ids", torch.int32, T * k, dev, k), _arg(topk_weights, "topk_weights", f32, T * k, dev, k),
               _arg(dweights, "dweights", f32, T * k, dev, k), bp, dp)


def moe_sort_workspace_bytes(n: int, n_experts: int) -> int:
    b = C.c_size_t()
    _check(lib().moe_sort_workspace_bytes(_int32(n, "n"), _int32(n_experts, "n_experts"), C.byref(b)))
    return b.value


def moe_sort_assignments(ids, n_experts, expert_counts, expert_offsets, sorted_assign, ws, stream=None):
    """int32 ids (any shape) -> expert_counts [E], expert_offsets [E + 1], sorted_assign [ids.numel()] int32."""
    torch = _torch()
    n, E, i32, dev = _int32(ids.numel(), "the number of ids"), _int32(n_experts, "n_experts"), torch.int32, ids.get_device()
    _on_device(dev, stream, lib().moe_sort_assignments, _arg(ids, "ids", i32, n, dev), n, E,
               _arg(expert_counts, "expert_counts", i32, E, dev), _arg(expert_offsets, "expert_offsets", i32, E + 1, dev),
               _arg(sorted_assign, "sorted_assign", i32, n, dev), *_bytes(ws, dev))


def _combine_shape(rows, y, name, *by_place):
    """(T, k, width, device index) from rows [T * k, width] and y or dy [T, width]; without tokens k is that of the first
    [T, k] tensor."""
    if rows.dim() != 2 or y.dim() != 2:
        _bad(f"rows and {name} must be 2-D (got {tuple(rows.shape)}, {tuple(y.shape)})")
    n, (T, width) = rows.shape[0], y.shape
    if T:
        k = n // T
    else:
        k = next((t.shape[-1] for t in by_place if t is not None and t.dim() > 1), 1)
    if n != T * k:
        _bad(f"rows must be [T * k, width] and {name} [T, width] (got {tuple(rows.shape)}, {tuple(y.shape)})")
    return _int32(T, "T"), _int32(k, "k"), _int32(width, "width"), y.get_device()


def moe_combine_forward(rows, topk_ids, weights, base, y, stream=None):
    """y [T, width] = base (or zeros) + the sum over j of weights[t, j] * rows[t * k + j], without the rows whose id is
    negative; rows [T * k, width], topk_ids [T, k] int32 or None, weights [T, k] float32 or None (1)."""
    torch = _torch()
    T, k, H, dev = _combine_shape(rows, y, "y", topk_ids, weights)
    rows_kind, rp = _matrix(rows, "rows", T * k, H, dev)
    kind, yp = _matrix(y, "y", T, H, dev)
    base_kind, bp = _matrix(base, "base", T, H, dev)
    _same_type(base_kind, kind, "base and y")
    ids = None if topk_ids is None else _arg(topk_ids, "topk_ids", torch.int32, T * k, dev, k)
    w = None if weights is None else _arg(weights, "weights", torch.float32, T * k, dev, k)
    _on_device(dev, stream, lib().moe_combine_forward, rp, rows_kind, T, k, H, ids, w, bp, yp, kind)


def moe_combine_backward(dy, rows, topk_ids, weights, drows, dweights, stream=None):
    """The gradients drows [T * k, width] (of rows' type) and dweights [T, k] float32 for dy [T, width]; either may be
    None, and rows where dweights is."""
    torch = _torch()
    like = rows if rows is not None else drows
    if like is None:
        _bad("rows is missing" if dweights is not None else "drows and dweights are both missing")
    T, k, H, dev = _combine_shape(like, dy, "dy", topk_ids, weights, dweights)
    kind, dp = _matrix(dy, "dy", T, H, dev)
    rows_kind, rp = _matrix(rows, "rows", T * k, H, dev)
    drows_kind, drp = _matrix(drows, "drows", T * k, H, dev)
    if rows_kind is None:
        rows_kind = drows_kind
    _same_type(drows_kind, rows_kind, "drows and rows")
    ids = None if topk_ids is None else _arg(topk_ids, "topk_ids", torch.int32, T * k, dev, k)
    w = None if weights is None else _arg(weights, "weights", torch.float32, T * k, dev, k)
    dw = None if dweights is None else _arg(dweights, "dweights", torch.float32, T * k, dev, k)
    _on_device(dev, stream, lib().moe_combine_backward, dp, kind, rp, rows_kind, T, k, H, ids, w, drp, dw)


def make_adapter_desc(n_adapters, rank, n_in, n_out, y_type) -> AdapterDesc:
    return AdapterDesc(_int32(n_adapters, "n_adapters"), _int32(rank, "rank"), _int32(n_in, "n_in"), _int32(n_out, "n_out"),
                       y_type)


def moe_adapters_workspace_bytes(desc, rows: int) -> int:
    n = C.c_size_t()
    _check(lib().moe_adapters_workspace_bytes(C.byref(desc), _int32(rows, "rows"), C.byref(n)))
    return n.value


def _adapter_args(desc, a, b, scales, x, offsets, rows, src_rows, src_div, dst_rows):
    """What both directions take alike: (device index, rows, src_div, x's rows), (a, b, scales, x), (offsets, src_rows,
    dst_rows)."""
    torch = _torch()
    n, r, K, N = desc.n_adapters, desc.rank, desc.n_in, desc.n_out
    dev, bf16, i32 = x.get_device(), torch.bfloat16, torch.int32
    if desc.y_type not in (MOE_F32, MOE_BF16):
        _bad(f"y_type must be MOE_F32 or MOE_BF16 (got {desc.y_type})")
    if x.dim() != 2 or x.shape[1] != K:
        _bad(f"x must be 2-D with {K} columns (got {tuple(x.shape)})")
    rows, src_div, x_rows = _int32(rows, "rows"), _int32(src_div, "src_div"), _int32(x.shape[0], "the number of x's rows")
    return ((dev, rows, src_div, x_rows),
            (_arg(a, "a", bf16, n * r * K, dev, K), _arg(b, "b", bf16, n * N * r, dev, r),
             None if scales is None else _arg(scales, "scales", torch.float32, n, dev), _arg(x, "x", bf16, x_rows * K, dev)),
            (_arg(offsets, "offsets", i32, n + 1, dev), None if src_rows is None else _arg(src_rows, "src_rows", i32, rows, dev),
             None if dst_rows is None else _arg(dst_rows, "dst_rows", i32, rows, dev)))


def _adapter_rows(desc, t, name, dev):
    """(rows, address) of y or dy."""
    if t.dim() != 2:
        _bad(f"{name} must be 2-D (got {tuple(t.shape)})")
    kind, p = _matrix(t, name, t.shape[0], desc.n_out, dev)
    if kind != desc.y_type:
        _bad(f"{name} must have the descriptor's y_type (got {t.dtype})")
    return _int32(t.shape[0], f"the number of {name}'s rows"), p


def moe_adapters_forward(desc, a, b, scales, x, offsets, rows, base, y, h=None, src_rows=None, src_div=1, dst_rows=None,
                         stream=None):
    """Position i of adapter e's range gives y[dst_rows[i]] = base (or zeros) + scales[e] * b[e] (a[e] x[src_rows[i] //
    src_div]); a [n, rank, n_in], b [n, n_out, rank], x bfloat16, scales [n] float32 or None, h [rows, rank] float32 or
    None: a[e] x by position, for the backward call."""
    (dev, rows, src_div, x_rows), factors, (off, src, dst) = _adapter_args(desc, a, b, scales, x, offsets, rows, src_rows,
                                                                           src_div, dst_rows)
    y_rows, yp = _adapter_rows(desc, y, "y", dev)
    base_kind, bp = _matrix(base, "base", y_rows, desc.n_out, dev)
    _same_type(base_kind, desc.y_type, "base and y")
    hp = None if h is None else _arg(h, "h", _torch().float32, rows * desc.rank, dev, desc.rank)
    _on_device(dev, stream, lib().moe_adapters_forward, C.byref(desc), *factors, x_rows, off, rows, src, src_div, dst, bp, yp,
               y_rows, hp)


def moe_adapters_backward(desc, a, b, scales, x, h, dy, offsets, rows, base, dx, da, db, ws=None, src_rows=None, src_div=1,
                          dst_rows=None, stream=None):
    """The gradients for dy: dx [x's rows * src_div (without src_rows x's rows), n_in] bfloat16 = base (or zeros) + ..., da
    [n, rank, n_in] and db [n, n_out, rank] float32; dx (with base) and da with db may be None."""
    torch = _torch()
    (dev, rows, src_div, x_rows), factors, (off, src, dst) = _adapter_args(desc, a, b, scales, x, offsets, rows, src_rows,
                                                                           src_div, dst_rows)
    n, r, K, N = desc.n_adapters, desc.rank, desc.n_in, desc.n_out
    y_rows, dyp = _adapter_rows(desc, dy, "dy", dev)
    dx_rows = x_rows * (src_div if src_rows is not None else 1)
    bf16, f32 = torch.bfloat16, torch.float32
    _on_device(dev, stream, lib().moe_adapters_backward, C.byref(desc), *factors, x_rows,
               None if h is None else _arg(h, "h", f32, rows * r, dev, r), dyp, y_rows, off, rows, src, src_div, dst,
               None if base is None else _arg(base, "base", bf16, dx_rows * K, dev, K),
               None if dx is None else _arg(dx, "dx", bf16, dx_rows * K, dev, K),
               None if da is None else _arg(da, "da", f32, n * r * K, dev, K),
               None if db is None else _arg(db, "db", f32, n * N * r, dev, r), *_bytes(ws, dev))


def make_desc(hidden, n_experts, top_k, inter, shared_inter, gemv_max_rows=-1, max_chunk=2048,
              tile_rows=0, group_size=64, host_sync_routing=0, dequant_pass=0, batch_invariant=0) -> LayerDesc:
    return LayerDesc(hidden, n_experts, top_k, inter, shared_inter, group_size, gemv_max_rows,
                     max_chunk, tile_rows, host_sync_routing, dequant_pass, batch_invariant)


def moe_packed_bytes(desc: LayerDesc) -> int:
    n = C.c_size_t()
    _check(lib().moe_packed_bytes(C.byref(desc), C.byref(n)))
    return n.value


def moe_workspace_bytes(desc: LayerDesc, max_tokens: int) -> int:
    n = C.c_size_t()
    _check(lib().moe_workspace_bytes(C.byref(desc), max_tokens, C.byref(n)))
    return n.value


def moe_max_tiles(desc: LayerDesc, T: int) -> int:
    n = C.c_int32()
    _check(lib().moe_max_tiles(C.byref(desc), T, C.byref(n)))
    return n.value


def moe_default_gemv_max_rows() -> int:
    return lib().moe_default_gemv_max_rows()


def _qm(m):
    if m is None:
        return QMatrix(None, None, None)
    codes, scales, biases = m
    return QMatrix(_ptr(codes), _ptr(scales), _ptr(biases))


def moe_pack_weights(desc, gate, up, down, sh_gate, sh_up, sh_down, packed, stream=None):
    """gate/up/down/sh_* are (codes, scales, biases) device tensors; packed a device byte tensor."""
    _check(lib().moe_pack_weights(C.byref(desc), _qm(gate), _qm(up), _qm(down), _qm(sh_gate),
                                  _qm(sh_up), _qm(sh_down), _ptr(packed),
                                  packed.numel() * packed.element_size(), _stream(stream)))


def moe_route(desc, x, T, router_w, logit_bias, routing: dict, ws, stream=None):
    """routing: dict of device tensors keyed like the moe_routing fields."""
    r = Routing(*(_ptr(routing[n]) for n, _ in Routing._fields_))
    _check(lib().moe_route(C.byref(desc), _ptr(x), T, _ptr(router_w), _ptr(logit_bias), C.byref(r),
                           _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_forward_prefill(desc, packed, router_w, logit_bias, x, T, y, ws, stream=None):
    _check(lib().moe_forward_prefill(C.byref(desc), _ptr(packed), _ptr(router_w), _ptr(logit_bias),
                                     _ptr(x), T, _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream)))


def moe_forward_decode(desc, packed, router_w, logit_bias, x, T, y, ws, stream=None):
    _check(lib().moe_forward_decode(C.byref(desc), _ptr(packed), _ptr(router_w), _ptr(logit_bias),
                                    _ptr(x), T, _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)))


def moe_forward_decode_static(desc, packed, router_w, logit_bias, x, T, y, stream=None):
    """moe_forward_decode on the library's fixed device scratch (no workspace argument)."""
    _check(lib().moe_forward_decode_static(C.byref(desc), _ptr(packed), _ptr(router_w), _ptr(logit_bias),
                                           _ptr(x), T, _ptr(y), _stream(stream)))


def moe_probe_stream_read(src, nbytes, sink, max_workgroups, stream=None):
    """Streaming read of nbytes of src (16-byte pieces per lane); sink holds max_workgroups words."""
    _check(lib().moe_probe_stream_read(_ptr(src), nbytes, _ptr(sink), max_workgroups, _stream(stream)))


def moe_probe_mfma_rate(iters, workgroups, clocks, sink, stream=None):
    """MFMA-only kernel: workgroups x 4 waves x iters x 8 MFMAs of 32x32x16 (32768 flop each)."""
    _check(lib().moe_probe_mfma_rate(iters, workgroups, _ptr(clocks), _ptr(sink), _stream(stream)))


def moe_profile_enable(mask: int):
    """Bit i set = record events around kernel id i (0 = off)."""
    _check(lib().moe_profile_enable(int(mask)))


def moe_profile_reset():
    _check(lib().moe_profile_reset())


def moe_profile_read(kernel_id: int):
    ms = C.c_double()
    n = C.c_int32()
    _check(lib().moe_profile_read(kernel_id, C.byref(ms), C.byref(n)))
    return ms.value, n.value
