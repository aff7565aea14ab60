"""Python binding of the AdaHOP GEMM library (libadahop.so, HIP for gfx950).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. PyTorch supplies device memory and the current stream. The functions
carry the C ABI's names (see include/adahop.h for the contract of each).

bf16 tensors may be passed as torch.bfloat16 or as int16 bit patterns.
There is no CPU fallback: if the library is missing this module raises.
"""
import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libadahop.so")

PAT = {"N": 0, "R": 1, "C": 2}
OP = {"FWD": 0, "DGRAD": 1, "WGRAD": 2}
ROUTE = {"AUTO": -1, "BF16": 0, "IHT": 1, "OE_LEFT": 2, "OE_RIGHT": 3, "OE_INNER": 4, "MXFP4": 5}
ROUTE_NAME = {v: k for k, v in ROUTE.items()}
AXIS = {"ROWS": 0, "COLS": 1}
OUT = {torch.bfloat16: 0, torch.float32: 1}
STAGE_EVENTS = 7
STAGES = ("foid", "quant_lhs", "quant_rhs", "oe_product", "gemm", "gemm_tail")

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_int = ctypes.c_int
_sz = ctypes.c_size_t


class AdahopError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"adahop status {status}: {detail}")


class MxOperand(ctypes.Structure):
    _fields_ = [("codes", _p), ("scales", _p), ("outer", _i64), ("K", _i64)]


class Bf16View(ctypes.Structure):
    _fields_ = [("ptr", _p), ("ld", _i64), ("inner_contiguous", _i32), ("reserved", _i32)]


class OeDesc(ctypes.Structure):
    _fields_ = [("route", _int), ("k", _i32), ("idx", _p), ("a", Bf16View), ("b", Bf16View)]


class Plan(ctypes.Structure):
    _fields_ = [("route", _int), ("m", _i64), ("n", _i64), ("K", _i64), ("k", _i32),
                ("scan_tensor", _i32), ("scan_axis", _int), ("layout", _int),
                ("ws_bytes", _sz), ("off_idx", _sz), ("off_a_codes", _sz),
                ("off_a_scales", _sz), ("off_b_codes", _sz), ("off_b_scales", _sz),
                ("off_lhs_lines", _sz), ("off_rhs_lines", _sz), ("oe_in_quant", _i32)]


class GemmOptions(ctypes.Structure):
    _fields_ = [("oe_in_quant", _i32), ("reserved", _i32 * 7)]


class CtxPlan(ctypes.Structure):
    _fields_ = [("route", _int), ("T", _i64), ("Din", _i64), ("Dout", _i64), ("k", _i32),
                ("layout", _int), ("ctx_bytes", _sz), ("off_idx", _sz), ("off_codes", _sz),
                ("off_scales", _sz), ("off_lines", _sz), ("save_ws_bytes", _sz),
                ("wgrad_ws_bytes", _sz)]


class RmsnormArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("x", _p), ("ld_x", _i64),
                ("residual", _p), ("ld_residual", _i64), ("gain", _p), ("h", _p), ("ld_h", _i64),
                ("y", _p), ("ld_y", _i64), ("codes", _p), ("ld_codes", _i64),
                ("scales", _p), ("ld_scales", _i64), ("rstd", _p),
                ("x_dtype", _i32), ("residual_dtype", _i32), ("gain_dtype", _i32),
                ("eps", ctypes.c_float), ("reserved", _i32 * 4)]


class RmsnormBackwardArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("dy", _p), ("ld_dy", _i64), ("h", _p),
                ("ld_h", _i64), ("gain", _p), ("rstd", _p), ("dh", _p), ("ld_dh", _i64),
                ("dx", _p), ("ld_dx", _i64), ("dgain", _p), ("dy_dtype", _i32),
                ("h_dtype", _i32), ("gain_dtype", _i32), ("reserved", _i32 * 5)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("m", _i64), ("N", _i64), ("K", _i64),
                ("a_codes", _p), ("ld_a_codes", _i64), ("a_scales", _p), ("ld_a_scales", _i64),
                ("b_codes", _p), ("ld_b_codes", _i64), ("b_scales", _p), ("ld_b_scales", _i64),
                ("bias", _p), ("residual", _p), ("ld_residual", _i64), ("out", _p),
                ("ld_out", _i64), ("out_scales", _p), ("ld_out_scales", _i64), ("z", _p),
                ("ld_z", _i64), ("b_format", _i32), ("bias_dtype", _i32), ("act", _i32),
                ("gated", _i32), ("products", _i32), ("reserved", _i32 * 3)]


# Exported symbols and their C signatures (argtypes, restype).
SIGNATURES = {
    "adahop_status_string": ([_int], ctypes.c_char_p),
    "adahop_last_error": ([], ctypes.c_char_p),
    "adahop_version": ([], _int),
    "adahop_route": ([_int, _int, _int], _int),
    "adahop_detect_workspace_size": ([_i64, _i64, _int, _i32], _sz),
    "adahop_detect": ([_p, _i64, _i64, _i64, _int, _i32, _i32, _p, _p, _sz, _p], _int),
    "adahop_detect_noalloc_max_bytes": ([], _sz),
    "adahop_detect_noalloc": ([_p, _i64, _i64, _i64, _int, _i32, _i32, _p, _p], _int),
    "adahop_line_scores": ([_p, _i64, _i64, _i64, _int, _i32, _p, _p], _int),
    "adahop_classify_pattern": ([ctypes.POINTER(ctypes.c_double), _i64,
                                 ctypes.POINTER(ctypes.c_double), _i64, ctypes.c_double], _int),
    "adahop_iht_quant": ([_p, _i64, _i64, _i64, _int, _i32, _p, _i32, _int, _p, _p, _p, _p],
                         _int),
    "adahop_gemm_mx_workspace_size": ([_i64, _i64, _i64, ctypes.POINTER(OeDesc)], _sz),
    "adahop_gemm_mx": ([ctypes.POINTER(MxOperand), ctypes.POINTER(MxOperand),
                        ctypes.POINTER(OeDesc), _p, _i64, _int, _p, _sz, _p], _int),
    "adahop_gemm_plan": ([_int, _i64, _i64, _i64, _int, _int, _int, _i32,
                          ctypes.POINTER(Plan)], _int),
    "adahop_gemm_workspace_size": ([_int, _i64, _i64, _i64, _int, _int, _int, _i32], _sz),
    "adahop_gemm": ([_int, _p, _p, _i64, _i64, _i64, _int, _int, _int, _i32, _p, _int, _p,
                     _sz, _p], _int),
    "adahop_gemm_timed": ([_int, _p, _p, _i64, _i64, _i64, _int, _int, _int, _i32, _p, _int,
                           _p, _sz, _p, _p], _int),
    "adahop_gemm_plan_ex": ([_int, _i64, _i64, _i64, _int, _int, _int, _i32,
                             ctypes.POINTER(GemmOptions), ctypes.POINTER(Plan)], _int),
    "adahop_gemm_ex": ([_int, _p, _p, _i64, _i64, _i64, _int, _int, _int, _i32,
                        ctypes.POINTER(GemmOptions), _p, _int, _p, _sz, _p, _p], _int),
    "adahop_ctx_plan": ([_i64, _i64, _i64, _int, _int, _int, _i32, ctypes.POINTER(CtxPlan)], _int),
    "adahop_ctx_save": ([_p, _i64, _i64, _i64, _int, _int, _int, _i32, _p, _sz, _p, _sz, _p],
                        _int),
    "adahop_gemm_wgrad_ctx": ([_p, _p, _sz, _i64, _i64, _i64, _int, _int, _int, _i32, _p, _int,
                               _p, _sz, _p, _p], _int),
    "adahop_mx8_quant": ([_p, _int, _i64, _i64, _i64, _p, _i64, _p, _i64, _p], _int),
    "adahop_mx8_dequant": ([_p, _i64, _p, _i64, _i64, _i64, _p, _int, _i64, _p], _int),
    "adahop_rmsnorm": ([ctypes.POINTER(RmsnormArgs), _p], _int),
    "adahop_rmsnorm_backward_workspace_size": ([_i64, _i64], _sz),
    "adahop_rmsnorm_backward": ([ctypes.POINTER(RmsnormBackwardArgs), _p, _sz, _p], _int),
    "adahop_linear_mx_workspace_size": ([_i64, _i64, _i64, _int, _i32], _sz),
    "adahop_linear_mx_args_workspace_size": ([ctypes.POINTER(LinearArgs)], _sz),
    "adahop_linear_mx": ([ctypes.POINTER(LinearArgs), _p, _sz, _p], _int),
    "adahop_act_backward_workspace_size": ([_i64, _i64, _i32], _sz),
    "adahop_act_backward": ([_p, _int, _i64, _p, _i64, _i64, _i64, _int, _i32, _p, _i64, _p, _p,
                             _sz, _p], _int),
}

_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "python -c 'import __graft_entry__ as g; g.build()'")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _check(status: int):
    if status != 0:
        raise AdahopError(status, lib().adahop_last_error().decode())


def _stream(device=None) -> int:
    """The current stream's handle (without a Stream object: 0.1 us for 2).
    Host tensors end here at the latest: the library would launch on their
    addresses."""
    if device is not None and device.type != "cuda":
        raise ValueError(f"expected a GPU device, got {device}")
    index = None if device is None else device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def _bf16_ptr(t: torch.Tensor, name: str) -> int:
    if t.dtype not in (torch.bfloat16, torch.int16):
        raise TypeError(f"{name}: expected bfloat16 (or int16 bit patterns), got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name}: expected a 2-D tensor with unit column stride")
    return t.data_ptr()


def _on_device(device: torch.device, **tensors):
    """Every tensor that is given lies on `device`, a GPU."""
    if device.type != "cuda":
        raise ValueError(f"expected GPU tensors, got {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name}: on {t.device}, the other operands on {device}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _axis(a) -> int:
    return AXIS[a] if isinstance(a, str) else int(a)


def adahop_route(op: str, pat_lhs: str, pat_rhs: str) -> str:
    r = lib().adahop_route(OP[op], PAT[pat_lhs], PAT[pat_rhs])
    if r == ROUTE["AUTO"]:
        raise ValueError("invalid op or pattern")
    return ROUTE_NAME[r]


def adahop_detect_workspace_size(rows: int, cols: int, axis, k: int) -> int:
    return lib().adahop_detect_workspace_size(rows, cols, _axis(axis), k)


def adahop_detect(t: torch.Tensor, axis, k: int, probe: int = 64,
                  idx_out: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """FOID: int32 [k] indices of the outlier rows/columns of t, ascending."""
    ptr = _bf16_ptr(t, "t")
    rows, cols = t.shape
    if idx_out is None:
        idx_out = torch.empty(max(k, 1), dtype=torch.int32, device=t.device)
    need = adahop_detect_workspace_size(rows, cols, axis, k)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=t.device)
    _check(lib().adahop_detect(ptr, rows, cols, t.stride(0), _axis(axis), probe, k,
                               idx_out.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
                               _stream(t.device)))
    return idx_out[:k]


def adahop_detect_noalloc(t: torch.Tensor, axis, k: int, probe: int = 64,
                          idx_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """FOID with the library's static scratch (no workspace): int32 [k]
    indices, ascending. Pass idx_out to keep the call free of allocation."""
    ptr = _bf16_ptr(t, "t")
    rows, cols = t.shape
    if idx_out is None:
        idx_out = torch.empty(max(k, 1), dtype=torch.int32, device=t.device)
    _check(lib().adahop_detect_noalloc(ptr, rows, cols, t.stride(0), _axis(axis), probe, k,
                                       idx_out.data_ptr(), _stream(t.device)))
    return idx_out[:k]


def adahop_line_scores(t: torch.Tensor, axis, probe: int = 64,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """FOID's score of every row (axis ROWS) or column (COLS) of t: fp64 on the device."""
    ptr = _bf16_ptr(t, "t")
    rows, cols = t.shape
    n = rows if _axis(axis) == AXIS["ROWS"] else cols
    if out is None:
        out = torch.empty(n, dtype=torch.float64, device=t.device)
    _check(lib().adahop_line_scores(ptr, rows, cols, t.stride(0), _axis(axis), probe,
                                    out.data_ptr(), _stream(t.device)))
    return out


CLASSIFY_THRESHOLD = 8.0


def adahop_classify_pattern(row_scores, col_scores, threshold: float = CLASSIFY_THRESHOLD) -> str:
    """"R", "C" or "N" from a tensor's row and column scores (host copies are made)."""
    r = np.ascontiguousarray(torch.as_tensor(row_scores).detach().cpu().numpy(), dtype=np.float64)
    c = np.ascontiguousarray(torch.as_tensor(col_scores).detach().cpu().numpy(), dtype=np.float64)
    dp = ctypes.POINTER(ctypes.c_double)
    p = lib().adahop_classify_pattern(r.ctypes.data_as(dp), r.size, c.ctypes.data_as(dp), c.size,
                                      float(threshold))
    return {v: k for k, v in PAT.items()}[p]


def adahop_calibrate(t: torch.Tensor, probe: int = 64,
                     threshold: float = CLASSIFY_THRESHOLD) -> str:
    """The pattern of a bf16 tensor from its row and column scores."""
    rs = adahop_line_scores(t, "ROWS", probe)
    cs = adahop_line_scores(t, "COLS", probe)
    return adahop_classify_pattern(rs, cs, threshold)


def adahop_iht_quant(src: torch.Tensor, contract, hadamard_block: int = 32,
                     zero_idx: Optional[torch.Tensor] = None, zero_axis="ROWS",
                     gather: bool = True):
    """(codes [outer][K/2] u8, scales [outer][K/32] u8, gathered bf16 or None)."""
    ptr = _bf16_ptr(src, "src")
    rows, cols = src.shape
    c = _axis(contract)
    K, outer = (cols, rows) if c == AXIS["COLS"] else (rows, cols)
    dev = src.device
    codes = torch.empty((outer, max(K // 2, 1)), dtype=torch.uint8, device=dev)
    scales = torch.empty((outer, max(K // 32, 1)), dtype=torch.uint8, device=dev)
    nz = 0 if zero_idx is None else zero_idx.numel()
    za = _axis(zero_axis)
    gathered = None
    if nz and gather:
        shape = (nz, cols) if za == AXIS["ROWS"] else (nz, rows)   # one line per row
        gathered = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if zero_idx is not None and zero_idx.dtype != torch.int32:
        raise TypeError("zero_idx must be int32")
    _check(lib().adahop_iht_quant(ptr, rows, cols, src.stride(0), c, hadamard_block,
                                  _ptr(zero_idx), nz, za, codes.data_ptr(), scales.data_ptr(),
                                  _ptr(gathered), _stream(dev)))
    return codes, scales, gathered


def bf16_view(t: torch.Tensor, inner_contiguous: bool) -> Bf16View:
    return Bf16View(_bf16_ptr(t, "view"), t.stride(0), int(inner_contiguous), 0)


def adahop_gemm_mx(a_codes, a_scales, b_codes, b_scales, oe: Optional[dict] = None,
                   out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None):
    """C = deq(A) deq(B)^T (+ the outlier term). oe: {"route", "k", "idx", "a":
    (tensor, inner_contiguous), "b": (tensor, inner_contiguous)}."""
    m, n, K = a_codes.shape[0], b_codes.shape[0], a_codes.shape[1] * 2
    A = MxOperand(a_codes.data_ptr(), a_scales.data_ptr(), m, K)
    B = MxOperand(b_codes.data_ptr(), b_scales.data_ptr(), n, b_codes.shape[1] * 2)
    dev = a_codes.device
    _on_device(dev, a_scales=a_scales, b_codes=b_codes, b_scales=b_scales, out=out,
               **({} if oe is None else {"oe idx": oe.get("idx"), "oe a": oe["a"][0], "oe b": oe["b"][0]}))
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
    desc = None
    ws = None
    if oe is not None:
        idx = oe.get("idx")
        desc = OeDesc(ROUTE[oe["route"]], oe["k"], _ptr(idx), bf16_view(*oe["a"]),
                      bf16_view(*oe["b"]))
    need = lib().adahop_gemm_mx_workspace_size(
        m, n, K, ctypes.byref(desc) if desc is not None else None)
    if need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().adahop_gemm_mx(ctypes.byref(A), ctypes.byref(B),
                                ctypes.byref(desc) if desc is not None else None,
                                out.data_ptr(), out.stride(0), OUT[out.dtype], _ptr(ws),
                                0 if ws is None else ws.numel(), _stream(dev)))
    return out


def _options(oe_in_quant: bool):
    return GemmOptions(oe_in_quant=1 if oe_in_quant else 0)


def adahop_gemm_plan(op: str, T: int, Din: int, Dout: int, pat_lhs="N", pat_rhs="N",
                     route: Optional[str] = None, oe_rank: int = 64,
                     oe_in_quant: bool = False) -> Plan:
    """The call's plan; oe_in_quant asks for the outlier product formed in
    the other operand's quantization (adahop_gemm_plan_ex)."""
    p = Plan()
    if oe_in_quant:
        o = _options(True)
        _check(lib().adahop_gemm_plan_ex(OP[op], T, Din, Dout, PAT[pat_lhs], PAT[pat_rhs],
                                         ROUTE[route or "AUTO"], oe_rank, ctypes.byref(o),
                                         ctypes.byref(p)))
    else:
        _check(lib().adahop_gemm_plan(OP[op], T, Din, Dout, PAT[pat_lhs], PAT[pat_rhs],
                                      ROUTE[route or "AUTO"], oe_rank, ctypes.byref(p)))
    return p


def adahop_gemm_workspace_size(op: str, T: int, Din: int, Dout: int, pat_lhs="N",
                               pat_rhs="N", route: Optional[str] = None,
                               oe_rank: int = 64) -> int:
    return adahop_gemm_plan(op, T, Din, Dout, pat_lhs, pat_rhs, route, oe_rank).ws_bytes


def _gemm_dims(op, lhs, rhs):
    if op == "FWD":
        (T, Din), (Dout, Din2) = lhs.shape, rhs.shape
        ok = Din == Din2
        out_shape = (T, Dout)
    elif op == "DGRAD":
        (T, Dout), (Dout2, Din) = lhs.shape, rhs.shape
        ok = Dout == Dout2
        out_shape = (T, Din)
    elif op == "WGRAD":
        (T, Dout), (T2, Din) = lhs.shape, rhs.shape
        ok = T == T2
        out_shape = (Dout, Din)
    else:
        raise ValueError(f"invalid op {op}")
    if not ok:
        raise ValueError(f"{op}: operand shapes {tuple(lhs.shape)} and {tuple(rhs.shape)} disagree")
    return T, Din, Dout, out_shape


def adahop_gemm(op: str, lhs: torch.Tensor, rhs: torch.Tensor, pat_lhs="N", pat_rhs="N",
                route: Optional[str] = None, oe_rank: int = 64, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stage_events: Optional[Sequence] = None, oe_in_quant: bool = False):
    """One AdaHOP product; returns the output tensor. `ws` (uint8, at least
    the planned size) is optional; after the call it holds the quantized
    operands at the offsets of adahop_gemm_plan. stage_events: STAGE_EVENTS
    torch.cuda.Event(enable_timing=True), recorded at the stage boundaries.
    oe_in_quant: form the outlier product in the other operand's
    quantization where it applies (adahop_gemm_ex)."""
    for t, nm in ((lhs, "lhs"), (rhs, "rhs")):
        _bf16_ptr(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    T, Din, Dout, out_shape = _gemm_dims(op, lhs, rhs)
    plan = adahop_gemm_plan(op, T, Din, Dout, pat_lhs, pat_rhs, route, oe_rank, oe_in_quant)
    dev = lhs.device
    if out is None:
        out = torch.empty(out_shape, dtype=out_dtype, device=dev)
    if ws is None and plan.ws_bytes:
        ws = torch.empty(plan.ws_bytes, dtype=torch.uint8, device=dev)
    args = [OP[op], lhs.data_ptr(), rhs.data_ptr(), T, Din, Dout, PAT[pat_lhs], PAT[pat_rhs],
            ROUTE[route or "AUTO"], oe_rank, out.data_ptr(), OUT[out.dtype], _ptr(ws),
            0 if ws is None else ws.numel(), _stream(dev)]
    handles = None
    if stage_events is not None:
        if len(stage_events) != STAGE_EVENTS:
            raise ValueError(f"stage_events needs {STAGE_EVENTS} events")
        handles = (ctypes.c_void_p * STAGE_EVENTS)(*[_event_handle(e) for e in stage_events])
    if oe_in_quant:
        o = _options(True)
        _check(lib().adahop_gemm_ex(*args[:10], ctypes.byref(o), *args[10:], handles))
    elif handles is None:
        _check(lib().adahop_gemm(*args))
    else:
        _check(lib().adahop_gemm_timed(*args, handles))
    return out


def _event_handle(ev: "torch.cuda.Event") -> int:
    # torch creates the underlying hipEvent lazily, at the first record().
    if ev.cuda_event == 0:
        ev.record()
    return ev.cuda_event


LAYOUT_ROWS, LAYOUT_KCHUNK = 0, 1


def unpack_packed(codes: torch.Tensor, scales: torch.Tensor, outer: int, K: int, layout: int):
    """Packed operand bytes in `layout` as row-major ([outer][K/2] codes,
    [outer][K/32] scales); a K-chunked operand is reordered (a copy)."""
    if layout == LAYOUT_KCHUNK:     # [K/128][outer][64], [K/128][outer][4]
        codes = codes.view(K // 128, outer, 64).permute(1, 0, 2).reshape(outer, K // 2)
        # a chunk's scale bytes are its blocks' in the order 0, 2, 1, 3
        scales = scales.view(K // 128, outer, 4)[:, :, [0, 2, 1, 3]]
        scales = scales.permute(1, 0, 2).reshape(outer, K // 32)
    return codes.view(outer, K // 2), scales.view(outer, K // 32)


def workspace_views(ws: torch.Tensor, plan: Plan) -> dict:
    """The intermediates a call leaves in its workspace, as tensors. Packed
    operands are returned in the row-major layout ([outer][K/2] codes,
    [outer][K/32] scales); a K-chunked plan's are reordered into it (a copy)."""
    none = (1 << 64) - 1
    m, n, K, k = plan.m, plan.n, plan.K, plan.k

    def region(off, count, dtype):
        if off == none:
            return None
        nbytes = count * torch.tensor([], dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype)

    def packed(off_codes, off_scales, outer):
        codes = region(off_codes, outer * (K // 2), torch.uint8)
        scales = region(off_scales, outer * (K // 32), torch.uint8)
        if codes is None:
            return None, None
        return unpack_packed(codes, scales, outer, K, plan.layout)

    out = {"idx": region(plan.off_idx, k, torch.int32)}
    out["a_codes"], out["a_scales"] = packed(plan.off_a_codes, plan.off_a_scales, m)
    out["b_codes"], out["b_scales"] = packed(plan.off_b_codes, plan.off_b_scales, n)
    return out


# ---------------------------------------------------------------------------
# Saved forward context of the activation X for the weight gradient
# ---------------------------------------------------------------------------
def adahop_ctx_plan(T: int, Din: int, Dout: int, pat_gy="N", pat_x="N",
                    route: Optional[str] = None, oe_rank: int = 64) -> CtxPlan:
    p = CtxPlan()
    _check(lib().adahop_ctx_plan(T, Din, Dout, PAT[pat_gy], PAT[pat_x], ROUTE[route or "AUTO"],
                                 oe_rank, ctypes.byref(p)))
    return p


def adahop_ctx_save(X: torch.Tensor, Dout: int, pat_gy="N", pat_x="N",
                    route: Optional[str] = None, oe_rank: int = 64,
                    ctx: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The context X [T, Din] keeps for its weight gradient (uint8 device
    buffer laid out as adahop_ctx_plan says)."""
    _bf16_ptr(X, "X")
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    T, Din = X.shape
    plan = adahop_ctx_plan(T, Din, Dout, pat_gy, pat_x, route, oe_rank)
    if ctx is None:
        ctx = torch.empty(max(plan.ctx_bytes, 1), dtype=torch.uint8, device=X.device)
    if ws is None and plan.save_ws_bytes:
        ws = torch.empty(plan.save_ws_bytes, dtype=torch.uint8, device=X.device)
    _check(lib().adahop_ctx_save(X.data_ptr(), T, Din, Dout, PAT[pat_gy], PAT[pat_x],
                                 ROUTE[route or "AUTO"], oe_rank, ctx.data_ptr(), ctx.numel(),
                                 _ptr(ws), 0 if ws is None else ws.numel(), _stream(X.device)))
    return ctx


def adahop_gemm_wgrad_ctx(GY: torch.Tensor, ctx: torch.Tensor, Din: int, pat_gy="N", pat_x="N",
                          route: Optional[str] = None, oe_rank: int = 64,
                          out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None,
                          stage_events: Optional[Sequence] = None) -> torch.Tensor:
    """dW [Dout, Din] = GY^T X with X taken from its saved context."""
    _bf16_ptr(GY, "GY")
    if not GY.is_contiguous():
        raise ValueError("GY must be contiguous")
    if ctx.dtype != torch.uint8 or not ctx.is_cuda:
        raise TypeError("ctx must be a uint8 device tensor")
    T, Dout = GY.shape
    plan = adahop_ctx_plan(T, Din, Dout, pat_gy, pat_x, route, oe_rank)
    if out is None:
        out = torch.empty((Dout, Din), dtype=out_dtype, device=GY.device)
    if ws is None and plan.wgrad_ws_bytes:
        ws = torch.empty(plan.wgrad_ws_bytes, dtype=torch.uint8, device=GY.device)
    handles = None
    if stage_events is not None:
        if len(stage_events) != STAGE_EVENTS:
            raise ValueError(f"stage_events needs {STAGE_EVENTS} events")
        handles = (ctypes.c_void_p * STAGE_EVENTS)(*[_event_handle(e) for e in stage_events])
    _check(lib().adahop_gemm_wgrad_ctx(GY.data_ptr(), ctx.data_ptr(), ctx.numel(), T, Din, Dout,
                                       PAT[pat_gy], PAT[pat_x], ROUTE[route or "AUTO"], oe_rank,
                                       out.data_ptr(), OUT[out.dtype], _ptr(ws),
                                       0 if ws is None else ws.numel(), _stream(GY.device),
                                       handles))
    return out


def ctx_views(ctx: torch.Tensor, plan: CtxPlan) -> dict:
    """The arrays of a saved context as tensors: idx [k] (or None), codes
    [Din][T/2] and scales [Din][T/32] row-major (reordered from K-chunked if
    needed), lines [k][T] bf16 bits (or None)."""
    none = (1 << 64) - 1
    T, Din, k = plan.T, plan.Din, plan.k
    codes = ctx[plan.off_codes:plan.off_codes + Din * T // 2]
    scales = ctx[plan.off_scales:plan.off_scales + Din * T // 32]
    c, sc = unpack_packed(codes, scales, Din, T, plan.layout)
    return {"idx": None if plan.off_idx == none else ctx[plan.off_idx:plan.off_idx + 4 * k].view(torch.int32),
            "codes": c, "scales": sc,
            "lines": None if plan.off_lines == none
            else ctx[plan.off_lines:plan.off_lines + 2 * k * T].view(torch.int16).view(k, T)}


# ---------------------------------------------------------------------------
# Around the products: norm, MXFP8, the linear layer with its epilogue, and
# their gradients
# ---------------------------------------------------------------------------
ACT = {"NONE": 0, "RELU": 1, "SILU": 2, "GELU": 3, "GELU_TANH": 4}
MX_FORMAT = {"MXFP4": 0, "MXFP8": 1}
PRODUCTS = {"AUTO": 0, "SCALED": 1, "EXACT": 2}
_FLOAT = {torch.bfloat16: 0, torch.int16: 0, torch.float32: 1}
_BF16 = {torch.bfloat16: 0, torch.int16: 0}
_CODES = {torch.uint8: 0, torch.float8_e4m3fn: 0}
_SCALES = {torch.uint8: 0, torch.float8_e8m0fnu: 0}


def _matrix(t: torch.Tensor, name: str, types: dict, rows: int, cols: int, device: int):
    """(address, leading dimension, type) of a 2-D device matrix of that size."""
    kind = types.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name}: unexpected dtype {t.dtype}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name}: must be on the same device as the other operands")
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: expected shape ({rows}, {cols}), got {tuple(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name}: expected unit column stride")
    return t.data_ptr(), (s0 if rows > 1 else cols), kind


def _vector(t: torch.Tensor, name: str, types: dict, n: int, device: int):
    kind = types.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name}: unexpected dtype {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: must be on the same device as the other operands")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: expected {n} contiguous elements")
    return t.data_ptr(), kind


def _size(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    return t.shape


def _scratch(need: int, ws: Optional[torch.Tensor], device):
    """(address, bytes, tensor) of the caller's workspace, or of a new one."""
    if ws is None:
        if not need:
            return None, 0, None
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError("ws: must be contiguous and on the same device as the operands")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def adahop_mx8_quant(src: torch.Tensor, codes: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes [rows, cols], scales [rows, cols / 32]), uint8, of a bf16 or fp32
    matrix in MXFP8."""
    rows, cols = _size(src, "src")
    dev = src.device
    if codes is None:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
    d = src.get_device()
    p, ld, kind = _matrix(src, "src", _FLOAT, rows, cols, d)
    c, ldc, _ = _matrix(codes, "codes", _CODES, rows, cols, d)
    sc, lds, _ = _matrix(scales, "scales", _SCALES, rows, cols // 32, d)
    _check(lib().adahop_mx8_quant(p, kind, rows, cols, ld, c, ldc, sc, lds, _stream(dev)))
    return codes, scales


def adahop_mx8_dequant(codes: torch.Tensor, scales: torch.Tensor, out_dtype=torch.bfloat16,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of an MXFP8 matrix, in bf16 (exact) or fp32."""
    rows, cols = _size(codes, "codes")
    dev = codes.device
    if out is None:
        out = codes.new_empty((rows, cols), dtype=out_dtype)
    d = codes.get_device()
    c, ldc, _ = _matrix(codes, "codes", _CODES, rows, cols, d)
    sc, lds, _ = _matrix(scales, "scales", _SCALES, rows, cols // 32, d)
    p, ld, kind = _matrix(out, "out", _FLOAT, rows, cols, d)
    _check(lib().adahop_mx8_dequant(c, ldc, sc, lds, rows, cols, p, kind, ld, _stream(dev)))
    return out


class RmsnormOut(NamedTuple):
    h: Optional[torch.Tensor]        # the new residual stream (None without a residual)
    y: Optional[torch.Tensor]        # bf16, if asked for
    codes: Optional[torch.Tensor]    # MXFP8, if asked for
    scales: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]     # fp32 [rows], if asked for


def adahop_rmsnorm(x: torch.Tensor, gain: torch.Tensor, residual: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, mx8: bool = True, bf16: bool = False,
                   save_rstd: bool = False, h: Optional[torch.Tensor] = None) -> RmsnormOut:
    """RMS norm of x (+ residual): h = x + residual in the residual's type,
    y = h / sqrt(mean h^2 + eps) * gain as MXFP8 codes and scales (mx8) and /
    or in bf16. h may be given (the residual itself, to update it in place)."""
    rows, cols = _size(x, "x")
    d = x.get_device()
    xp, ldx, xk = _matrix(x, "x", _FLOAT, rows, cols, d)
    gp, gk = _vector(gain, "gain", _FLOAT, cols, d)
    rp = hp = yp = cp = sp = tp = None
    ldr = ldh = rk = 0
    if residual is not None:
        rp, ldr, rk = _matrix(residual, "residual", _FLOAT, rows, cols, d)
        if h is None:
            h = residual.new_empty((rows, cols))
            hp, ldh = h.data_ptr(), cols
        else:
            if h.dtype != residual.dtype:
                raise TypeError("h must have the residual's dtype")
            hp, ldh, _ = _matrix(h, "h", _FLOAT, rows, cols, d)
    elif h is not None:
        raise ValueError("h goes with a residual")
    codes = scales = y = rstd = None
    if mx8:
        codes = x.new_empty((rows, cols), dtype=torch.uint8)
        scales = x.new_empty((rows, cols // 32), dtype=torch.uint8)
        cp, sp = codes.data_ptr(), scales.data_ptr()
    if bf16:
        y = x.new_empty((rows, cols), dtype=torch.bfloat16)
        yp = y.data_ptr()
    if save_rstd:
        rstd = x.new_empty(rows, dtype=torch.float32)
        tp = rstd.data_ptr()
    a = RmsnormArgs(rows, cols, xp, ldx, rp, ldr, gp, hp, ldh, yp, cols, cp, cols, sp, cols // 32, tp,
                    xk, rk, gk, eps)
    _check(lib().adahop_rmsnorm(ctypes.byref(a), _stream(x.device)))
    return RmsnormOut(h, y, codes, scales, rstd)


def adahop_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, gain: torch.Tensor,
                            rstd: torch.Tensor, dh: Optional[torch.Tensor] = None,
                            gain_grad: bool = True, dx: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None):
    """(dx, dgain): the gradient at h -- of x and of the residual alike -- from
    dy and, if given, the residual stream's dh; dgain is fp32 (None without
    gain_grad)."""
    rows, cols = _size(h, "h")
    dev, d = h.device, h.get_device()
    yp, ldy, yk = _matrix(dy, "dy", _FLOAT, rows, cols, d)
    hp, ldh, hk = _matrix(h, "h", _FLOAT, rows, cols, d)
    gp, gk = _vector(gain, "gain", _FLOAT, cols, d)
    rp, _ = _vector(rstd, "rstd", {torch.float32: 1}, rows, d)
    if dx is None:
        dx = torch.empty((rows, cols), dtype=h.dtype, device=dev)
    xp, ldx, xk = _matrix(dx, "dx", _FLOAT, rows, cols, d)
    a = RmsnormBackwardArgs(rows, cols, yp, ldy, hp, ldh, gp, rp, None, 0, xp, ldx, None, yk, hk, gk)
    if dh is not None:
        a.dh, a.ld_dh, ek = _matrix(dh, "dh", _FLOAT, rows, cols, d)
    if xk != hk or (dh is not None and ek != hk):
        raise TypeError("dx and dh must have h's dtype")
    dgain, wp, wn = None, None, 0
    if gain_grad:
        dgain = torch.empty(cols, dtype=torch.float32, device=dev)
        a.dgain = dgain.data_ptr()
        wp, wn, ws = _scratch(lib().adahop_rmsnorm_backward_workspace_size(rows, cols), ws, dev)
    _check(lib().adahop_rmsnorm_backward(ctypes.byref(a), wp, wn, _stream(dev)))
    return dx, dgain


class LinearOut(NamedTuple):
    out: torch.Tensor                # bf16, or MXFP8 codes
    scales: Optional[torch.Tensor]   # MXFP8 scales
    z: Optional[torch.Tensor]        # bf16 pre-activation, if asked for


def adahop_linear_mx(a: Tuple[torch.Tensor, torch.Tensor], b: Tuple[torch.Tensor, torch.Tensor],
                     bias: Optional[torch.Tensor] = None, act: str = "NONE", gated: bool = False,
                     residual: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                     save_z: bool = False, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, products: str = "AUTO") -> LinearOut:
    """act(z) + residual with z = A B^T + bias; gated: act(z[:, :n]) * z[:, n:].

    a: MXFP8 (codes [m, K], scales [m, K/32]); b: weights [N, K] in MXFP8, or
    in MXFP4 (codes [N, K/2], as adahop_iht_quant gives them). out_dtype:
    torch.bfloat16, or "MXFP8" for codes and scales. out (bf16) may be given,
    the residual itself among others. products: "EXACT", "SCALED" (faster on
    many rows; moves about one MXFP8 code in a thousand to its neighbour), or
    "AUTO": EXACT for MXFP8 outputs of up to 32768 values, else SCALED."""
    (ac, asc), (bc, bsc) = a, b
    m, K = _size(ac, "a codes")
    N, Kb = _size(bc, "b codes")
    dev, d = ac.device, ac.get_device()
    if Kb != K and Kb * 2 != K:
        raise ValueError(f"b codes: {Kb} bytes a row fit neither MXFP8 nor MXFP4 of K = {K}")
    n = N // 2 if gated else N
    fmt = 1 if Kb == K else 0
    ap, lda, _ = _matrix(ac, "a codes", _CODES, m, K, d)
    asp, ldas, _ = _matrix(asc, "a scales", _SCALES, m, K // 32, d)
    bp, ldb, _ = _matrix(bc, "b codes", _CODES, N, Kb, d)
    bsp, ldbs, _ = _matrix(bsc, "b scales", _SCALES, N, K // 32, d)
    biasp = rp = sp = zp = None
    bk = ldr = lds = 0
    if bias is not None:
        biasp, bk = _vector(bias, "bias", _FLOAT, N, d)
    if residual is not None:
        rp, ldr, _ = _matrix(residual, "residual", _BF16, m, n, d)
    scales = z = None
    if out_dtype == "MXFP8":
        if out is not None:
            raise ValueError("out is for a bf16 output")
        out = ac.new_empty((m, n), dtype=torch.uint8)
        scales = ac.new_empty((m, n // 32), dtype=torch.uint8)
        op, ldo, sp, lds = out.data_ptr(), n, scales.data_ptr(), n // 32
    elif out_dtype == torch.bfloat16:
        if out is None:
            out = ac.new_empty((m, n), dtype=torch.bfloat16)
            op, ldo = out.data_ptr(), n
        else:
            op, ldo, _ = _matrix(out, "out", _BF16, m, n, d)
    else:
        raise TypeError(f"out_dtype: torch.bfloat16 or \"MXFP8\", not {out_dtype}")
    if save_z:
        z = ac.new_empty((m, N), dtype=torch.bfloat16)
        zp = z.data_ptr()
    g = LinearArgs(m, N, K, ap, lda, asp, ldas, bp, ldb, bsp, ldbs, biasp, rp, ldr, op, ldo, sp, lds, zp, N,
                   fmt, bk, ACT[act], 1 if gated else 0, PRODUCTS[products])
    args = ctypes.byref(g)
    wp, wn, ws = _scratch(lib().adahop_linear_mx_args_workspace_size(args), ws, dev)
    _check(lib().adahop_linear_mx(args, wp, wn, _stream(dev)))
    return LinearOut(out, scales, z)


def adahop_act_backward(dout: torch.Tensor, z: torch.Tensor, act: str = "NONE", gated: bool = False,
                        bias_grad: bool = False, dz: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None):
    """(dz, dbias): the gradient of z [m, N] (bf16: the GY of adahop_gemm's
    DGRAD and WGRAD) and, if asked for, of the bias (fp32 [N])."""
    m, N = _size(z, "z")
    n = N // 2 if gated else N
    dev, d = z.device, z.get_device()
    gp, ldg, gk = _matrix(dout, "dout", _FLOAT, m, n, d)
    zp, ldz, _ = _matrix(z, "z", _BF16, m, N, d)
    if dz is None:
        dz = torch.empty((m, N), dtype=torch.bfloat16, device=dev)
    op, ldo, _ = _matrix(dz, "dz", _BF16, m, N, d)
    dbias, bp, wp, wn = None, None, None, 0
    if bias_grad:
        dbias = torch.empty(N, dtype=torch.float32, device=dev)
        bp = dbias.data_ptr()
        wp, wn, ws = _scratch(lib().adahop_act_backward_workspace_size(m, N, int(gated)), ws, dev)
    _check(lib().adahop_act_backward(gp, gk, ldg, zp, ldz, m, N, ACT[act], int(gated), op, ldo, bp, wp,
                                     wn, _stream(dev)))
    return dz, dbias
