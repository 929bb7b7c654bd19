"""Python binding of the MI355X sparse MoE FFN library (libmoe_gfx950.so).

Argument marshalling only: torch tensors provide device memory and the
current HIP stream; every step of the layer runs in the library's gfx950
kernels behind the C ABI declared in include/moe.h.  The library is loaded on
first use and a missing library is an error (there is no fallback path).

Entry points mirror the C ABI: route, permute, quant_e4m3_1x128,
quant_mxfp8, grouped_ffn, combine, layer, layer_noalloc (plus
workspace-size queries), and around the layer: ffn, ffn_backward, norm,
norm_backward, quant_i8, linear_i8.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_GFX950_LIB names another build of the same library (the host-sanitizer
# build the CPU tests run the boundary's argument checks under)
LIB_PATH = os.environ.get("MOE_GFX950_LIB") or os.path.join(HERE, "libmoe_gfx950.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
F32, BF16, E4M3, MXFP4, MXFP8, I8 = 0, 1, 2, 3, 4, 5
SOFTMAX, SIGMOID = 0, 1

DT = {"f32": F32, "bf16": BF16, "e4m3": E4M3, "mxfp4": MXFP4, "mxfp8": MXFP8, "i8": I8}
SCORE = {"softmax": SOFTMAX, "sigmoid": SIGMOID}

EXPORTS = [
    "moe_route", "moe_route_workspace_size", "moe_permute", "moe_permute_workspace_size",
    "moe_quant_e4m3_1x128", "moe_quant_mxfp8", "moe_grouped_ffn", "moe_grouped_ffn_workspace_size",
    "moe_combine", "moe_layer", "moe_layer_workspace_size", "moe_layer_noalloc", "moe_mx_pack_scales",
    "moe_ffn", "moe_ffn_workspace_size", "moe_ffn_backward", "moe_ffn_backward_workspace_size",
    "moe_norm", "moe_norm_backward", "moe_norm_backward_workspace_size",
    "moe_quant_i8", "moe_linear_i8", "moe_linear_i8_workspace_size",
    "moe_status_string", "moe_last_error",
]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_string(status)}: {msg}")
        self.status = status


class ExpertsT(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("dt", ctypes.c_int32),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("s_gate_up_packed", ctypes.c_void_p), ("s_down_packed", ctypes.c_void_p)]


_lib = None
_P, _I32, _SZ, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float


def lib() -> ctypes.CDLL:
    """Load libmoe_gfx950.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -m routed_expert_ffn_04_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_route": ([_P, _I32, _I32, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P], _I32),
            "moe_route_workspace_size": ([_I32, _I32], _SZ),
            "moe_permute": ([_P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P], _I32),
            "moe_permute_workspace_size": ([_I32, _I32, _I32], _SZ),
            "moe_quant_e4m3_1x128": ([_P, _I32, _I32, _I32, _P, _P, _P], _I32),
            "moe_quant_mxfp8": ([_P, _I32, _I32, _I32, _P, _P, _P], _I32),
            "moe_grouped_ffn": ([_P, _I32, _P, _P, _I32, _P, _I32, _I32, ctypes.POINTER(ExpertsT),
                                 _P, _P, _I32, ctypes.POINTER(ExpertsT), _P, _I32, _P, _P, _I32, _P, _SZ, _P], _I32),
            "moe_grouped_ffn_workspace_size": ([_I32, _I32, _I32, _I32, _I32, _I32], _SZ),
            "moe_combine": ([_P, _I32, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _P, _I32, _P], _I32),
            "moe_layer": ([_P, _I32, _I32, _I32, _P, _P, _I32, _I32, _I32, ctypes.POINTER(ExpertsT),
                           ctypes.POINTER(ExpertsT), _P, _I32, _I32, _P, _P, _P, _P, _SZ, _P], _I32),
            "moe_layer_workspace_size": ([_I32] * 10, _SZ),
            "moe_layer_noalloc": ([_P, _I32, _I32, _I32, _P, _P, _I32, _I32, _I32, ctypes.POINTER(ExpertsT),
                                   ctypes.POINTER(ExpertsT), _P, _I32, _I32, _P, _P, _P, _P], _I32),
            "moe_mx_pack_scales": ([ctypes.POINTER(ExpertsT), _P, _P, _P], _I32),
            "moe_ffn": ([_P, _I32, _I32, ctypes.POINTER(ExpertsT), _P, _I32, _P, _P, _SZ, _P], _I32),
            "moe_ffn_workspace_size": ([_I32] * 3, _SZ),
            "moe_ffn_backward": ([_P, _P, _I32, _I32, ctypes.POINTER(ExpertsT), _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
            "moe_ffn_backward_workspace_size": ([_I32] * 4, _SZ),
            "moe_norm": ([_P, _I32, _P, _I32, _I32, _I32, _P, _P, _I32, _P, _I32, _F32, _F32, _P, _P, _I32, _P, _P], _I32),
            "moe_norm_backward": ([_P, _I32, _P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _I32, _P, _I32, _F32, _F32,
                                   _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
            "moe_norm_backward_workspace_size": ([_I32] * 3, _SZ),
            "moe_quant_i8": ([_P, _I32, _I32, _I32, _P, _P, _P], _I32),
            "moe_linear_i8": ([_P, _P, _I32, _I32, _P, _P, _P, _I32, _P, _I32, _P, _SZ, _P], _I32),
            "moe_linear_i8_workspace_size": ([_I32] * 3, _SZ),
            "moe_status_string": ([_I32], ctypes.c_char_p),
            "moe_last_error": ([], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def status_string(st: int) -> str:
    return lib().moe_status_string(st).decode()


def _check(st: int):
    if st != MOE_OK:
        raise MoeError(st, lib().moe_last_error().decode())


# ---------------------------------------------------------------- helpers

def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dt_of(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _workspace(nbytes: int, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


@dataclass
class Experts:
    """Device tensors of an expert bank (output-major weights; see moe.h).
    dt: the weight type (default: from the tensor dtype; MXFP4 banks, packed
    uint8 [n][I][H/2] with uint8 E8M0 scales, must say MXFP4)."""
    w_gate: object
    w_up: object
    w_down: object
    s_gate: object = None
    s_up: object = None
    s_down: object = None
    dt: Optional[int] = None
    s_gate_up_packed: object = None    # MXFP4: exponents in the 16-row tiles' order (pack_mx_scales)
    s_down_packed: object = None

    def struct(self) -> ExpertsT:
        n, I, H = self.w_gate.shape
        dt = _dt_of(self.w_gate) if self.dt is None else self.dt
        if dt == MXFP4:
            H *= 2
        for t in (self.w_gate, self.w_up, self.w_down):
            assert t.is_contiguous() and t.is_cuda
        return ExpertsT(n, H, I, dt, _ptr(self.w_gate), _ptr(self.w_up), _ptr(self.w_down),
                        _ptr(self.s_gate), _ptr(self.s_up), _ptr(self.s_down),
                        _ptr(self.s_gate_up_packed), _ptr(self.s_down_packed))

    def pack_mx_scales(self, stream=None) -> "Experts":
        """A copy of this MXFP4 bank that also carries its exponents in the
        16-row tiles' order (moe_mx_pack_scales): a weight-load-time step.
        Returns the bank unchanged where the shape does not allow it
        (H % 1024 or I % 512 nonzero) or the weights are not MXFP4."""
        import dataclasses
        import torch
        st = self.struct()
        if st.dt != MXFP4 or st.H % 1024 or st.I % 512:
            return self
        dev = self.w_gate.device
        gu = torch.empty(2 * st.n * st.I * (st.H // 32), dtype=torch.uint8, device=dev)
        dn = torch.empty(st.n * st.H * (st.I // 32), dtype=torch.uint8, device=dev)
        _check(lib().moe_mx_pack_scales(ctypes.byref(st), _ptr(gu), _ptr(dn), _stream(stream)))
        return dataclasses.replace(self, s_gate_up_packed=gu, s_down_packed=dn)

    @staticmethod
    def from_bank(bank, pack: bool = True) -> "Experts":
        """Device bank of a synthetic bank; MXFP4 banks also get their packed
        exponents unless pack is False."""
        e = Experts(bank.w_gate, bank.w_up, bank.w_down, bank.s_gate, bank.s_up, bank.s_down,
                    MXFP4 if bank.dt == "mxfp4" else None)
        return e.pack_mx_scales() if pack and bank.dt == "mxfp4" else e


# ---------------------------------------------------------------- entry points

def route(x, w_router, bias, k: int, score: str, stream=None, ws=None, out=None):
    """topk_ids [T][k] int32, topk_w [T][k] fp32 (moe_route)."""
    import torch
    T, H = x.shape
    E = w_router.shape[1]
    if out is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    else:
        ids, w = out
    need = lib().moe_route_workspace_size(T, E)
    ws = ws if ws is not None else _workspace(need, x.device)
    _check(lib().moe_route(_ptr(x), _dt_of(x), T, H, _ptr(w_router), _ptr(bias), E, k, SCORE[score],
                           _ptr(ids), _ptr(w), _ptr(ws), ws.numel(), _stream(stream)))
    return ids, w


def permute(topk_ids, E: int, stream=None, ws=None, out=None):
    """counts [E], offsets [E+1], src [T*k], dest [T*k] (moe_permute)."""
    import torch
    T, k = topk_ids.shape
    dev = topk_ids.device
    if out is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        src = torch.empty(T * k, dtype=torch.int32, device=dev)
        dest = torch.empty(T * k, dtype=torch.int32, device=dev)
    else:
        counts, offsets, src, dest = out
    need = lib().moe_permute_workspace_size(T, k, E)
    ws = ws if ws is not None else _workspace(need, dev)
    _check(lib().moe_permute(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets), _ptr(src), _ptr(dest),
                             _ptr(ws), ws.numel(), _stream(stream)))
    return counts, offsets, src, dest


def quant_e4m3_1x128(x, stream=None, out=None):
    """codes [rows][cols] uint8, scales [rows][cols/128] fp32."""
    import torch
    rows, cols = x.shape
    if out is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        s = torch.empty((rows, cols // 128), dtype=torch.float32, device=x.device)
    else:
        q, s = out
    _check(lib().moe_quant_e4m3_1x128(_ptr(x), _dt_of(x), rows, cols, _ptr(q), _ptr(s), _stream(stream)))
    return q, s


def quant_mxfp8(x, stream=None, out=None):
    """MXFP8: E4M3 codes [rows][cols] uint8, E8M0 exponents [rows][cols/32] uint8."""
    import torch
    rows, cols = x.shape
    if out is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        e = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    else:
        q, e = out
    _check(lib().moe_quant_mxfp8(_ptr(x), _dt_of(x), rows, cols, _ptr(q), _ptr(e), _stream(stream)))
    return q, e


def _act_dt(a, a_scale) -> int:
    """E4M3 codes with fp32 1x128 scales, or MXFP8 codes with uint8 E8M0 exponents."""
    import torch
    if a_scale is not None and a_scale.dtype == torch.uint8:
        return MXFP8
    return _dt_of(a)


def _is_fp8(dtype) -> bool:
    import torch
    return dtype in (torch.uint8, torch.float8_e4m3fn)


def grouped_ffn(a, offsets, routed: Experts, *, a_scale=None, src=None, src_div: int = 1, R_max=None,
                a_sh=None, a_sh_scale=None, shared: Optional[Experts] = None, y_dtype=None,
                y=None, y_scale=None, y_sh=None, y_sh_dtype=None, stream=None, ws=None):
    """moe_grouped_ffn.  Returns (y [R_max][H], y_sh [S][H]); with an fp8 y_dtype
    (torch.uint8 codes) y is the pair (codes, scales [R_max][H/128])."""
    import torch
    rs = routed.struct()
    G, H = rs.n, rs.H
    R_max = (src.numel() if src is not None else a.shape[0]) if R_max is None else R_max
    S = 0 if a_sh is None else a_sh.shape[0]
    ss = shared.struct() if shared is not None else None
    y_dtype = y.dtype if y is not None else (y_dtype or torch.float32)
    fp8_y = _is_fp8(y_dtype)
    y_sh_dtype = y_sh_dtype or (torch.bfloat16 if fp8_y else y_dtype)
    dev = a.device
    if y is None:
        y = torch.empty((R_max, H), dtype=torch.uint8 if fp8_y else y_dtype, device=dev)
    if fp8_y and y_scale is None:
        y_scale = torch.empty((R_max, H // 128), dtype=torch.float32, device=dev)
    if y_sh is None and shared is not None and S > 0:
        y_sh = torch.empty((S, H), dtype=y_sh_dtype, device=dev)
    need = lib().moe_grouped_ffn_workspace_size(R_max, G, S if shared is not None else 0, H, rs.I, rs.dt)
    ws = ws if ws is not None else _workspace(need, dev)
    _check(lib().moe_grouped_ffn(_ptr(a), _act_dt(a, a_scale), _ptr(a_scale), _ptr(src), src_div, _ptr(offsets), G, R_max,
                                 ctypes.byref(rs), _ptr(a_sh), _ptr(a_sh_scale), S,
                                 ctypes.byref(ss) if ss is not None else None,
                                 _ptr(y), _dt_of(y), _ptr(y_scale) if fp8_y else None, _ptr(y_sh),
                                 _dt_of(y_sh) if y_sh is not None else F32, _ptr(ws), ws.numel(), _stream(stream)))
    return ((y, y_scale) if fp8_y else y), y_sh


def combine(y_perm, y_sh, dest, topk_w, out_dtype=None, out=None, stream=None, y_scale=None):
    """moe_combine.  y_perm fp32/bf16, or e4m3 codes (torch.uint8) with
    y_scale [rows][H/128]."""
    import torch
    T, k = topk_w.shape
    H = y_perm.shape[1]
    out_dtype = out_dtype or torch.float32
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=y_perm.device)
    _check(lib().moe_combine(_ptr(y_perm), _dt_of(y_perm), _ptr(y_scale), _ptr(y_sh),
                             _dt_of(y_sh) if y_sh is not None else F32, _ptr(dest), _ptr(topk_w), T, k, H,
                             _ptr(out), _dt_of(out), _stream(stream)))
    return out


def layer_workspace_size(T, H, E, k, I, x_dt, w_dt, has_shared, out_dt, y_dt=None) -> int:
    return lib().moe_layer_workspace_size(T, H, E, k, I, x_dt, w_dt, int(has_shared), out_dt,
                                          out_dt if y_dt is None else y_dt)


def layer(x, w_router, bias, k: int, score: str, routed: Experts, shared: Optional[Experts] = None,
          out_dtype=None, out=None, want_routing: bool = False, ws=None, stream=None, y_dtype=None):
    """The fused layer (moe_layer).  Returns out, or (out, ids, w, counts).
    y_dtype: dtype of the routed expert outputs before the combine (default:
    out_dtype; torch.uint8 = e4m3, the FP8 combine)."""
    import torch
    T, H = x.shape
    E = w_router.shape[1]
    rs = routed.struct()
    ss = shared.struct() if shared is not None else None
    out_dtype = out_dtype or torch.float32
    dev = x.device
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    ids = w = counts = None
    if want_routing:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
    y_dt = _dt_of(out) if y_dtype is None else (E4M3 if _is_fp8(y_dtype) else _dt_of(torch.empty(0, dtype=y_dtype)))
    need = layer_workspace_size(T, H, E, k, rs.I, _dt_of(x), rs.dt, ss is not None, _dt_of(out), y_dt)
    ws = ws if ws is not None else _workspace(need, dev)
    _check(lib().moe_layer(_ptr(x), _dt_of(x), T, H, _ptr(w_router), _ptr(bias), E, k, SCORE[score],
                           ctypes.byref(rs), ctypes.byref(ss) if ss is not None else None,
                           _ptr(out), _dt_of(out), y_dt, _ptr(ids), _ptr(w), _ptr(counts),
                           _ptr(ws), ws.numel(), _stream(stream)))
    return (out, ids, w, counts) if want_routing else out


def layer_noalloc(x, w_router, bias, k: int, score: str, routed: Experts, shared: Optional[Experts] = None,
                  out_dtype=None, out=None, want_routing: bool = False, stream=None, y_dtype=None):
    """moe_layer_noalloc: the fused layer with the library's own static
    scratch (no workspace argument, no device allocation by the library).
    Outputs are allocated here unless `out` (and, with want_routing, the
    routing buffers) are passed in."""
    import torch
    T, H = x.shape
    E = w_router.shape[1]
    rs = routed.struct()
    ss = shared.struct() if shared is not None else None
    out_dtype = out_dtype or torch.float32
    dev = x.device
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    ids = w = counts = None
    if want_routing:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        counts = torch.empty(E, dtype=torch.int32, device=dev)
    y_dt = _dt_of(out) if y_dtype is None else (E4M3 if _is_fp8(y_dtype) else _dt_of(torch.empty(0, dtype=y_dtype)))
    _check(lib().moe_layer_noalloc(_ptr(x), _dt_of(x), T, H, _ptr(w_router), _ptr(bias), E, k, SCORE[score],
                                   ctypes.byref(rs), ctypes.byref(ss) if ss is not None else None,
                                   _ptr(out), _dt_of(out), y_dt, _ptr(ids), _ptr(w), _ptr(counts), _stream(stream)))
    return (out, ids, w, counts) if want_routing else out


# ---------------------------------------------------------------- around the layer

torch = None        # imported by the first call below (the boundary itself does not need it)
_FLOATS = ()
_CODE = {}          # torch dtype -> moe_dtype_t


def _import_torch():
    global torch, _FLOATS, _CODE
    import torch as t
    _FLOATS = (t.float32, t.bfloat16)
    _CODE = {t.float32: F32, t.bfloat16: BF16, t.int8: I8}
    torch = t


# These calls are a few microseconds of GPU time at decode sizes, so what they do
# on the host is kept short: devices are compared by index, outputs are made
# by new_empty (quicker than torch.empty with a device), errors are put
# together only when there is one.

def _elsewhere(device: int, stream):
    """None if a call with tensors on GPU `device` can go to the current stream
    as it is, else the context in which it can: the device and `stream` (default:
    the device's current stream) made current, so that what the call allocates
    belongs to the stream that uses it."""
    if stream is None:
        if torch._C._cuda_getDevice() == device:
            return None
        stream = torch.cuda.current_stream(device)
    elif stream.device.index != device:
        raise ValueError(f"stream of {stream.device} with tensors on cuda:{device}")
    return torch.cuda.stream(stream)


def _current(device: int) -> int:
    """Handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device)


def _tensor(device: int, name, t, shape, dtypes):
    """Checks an argument (None passes): on the device, contiguous, of the
    shape and of one of the dtypes."""
    if t is None or (t.shape == shape and t.dtype in dtypes and t.get_device() == device and t.is_contiguous()):
        return
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    raise ValueError(f"{name} is not contiguous")


def _out_dtype(name, t, dtype, default):
    """dtype of an output: that of t, which `dtype` may repeat but not contradict."""
    if t is None:
        return dtype or default
    if dtype is not None and dtype is not t.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, but {dtype} is asked for")
    return t.dtype


def _empty(like, shape, dtype):
    """An output on `like`'s device."""
    if like.dtype is dtype:
        return torch.empty_like(like) if like.shape == shape else like.new_empty(shape)
    return like.new_empty(shape, dtype=dtype)


_MOST = 2 ** 31 - 1   # sizes cross the boundary as int32; ctypes would pass a larger one's low bits


def _matrix(name, t):
    """(rows, columns, device index) of a 2-d device tensor."""
    if torch is None:
        _import_torch()
    shape, device = t.shape, t.get_device()
    if len(shape) != 2 or device < 0:
        raise ValueError(f"{name}: expected a 2-d tensor on a GPU, got {tuple(shape)} on {t.device}")
    rows, columns = shape
    if rows > _MOST or columns > _MOST:
        raise ValueError(f"{name}: {tuple(shape)} has a size above {_MOST}")
    return rows, columns, device


def _scratch(ws, need, like):
    """(pointer, bytes) of the workspace given, or of a new one, and what keeps it alive."""
    if ws is None:
        need = max(need, 256)
        ws = like.new_empty(need, dtype=torch.uint8)
        return ws.data_ptr(), need, ws
    if ws.get_device() != like.get_device():
        raise ValueError(f"ws is on {ws.device}, expected {like.device}")
    if not ws.is_contiguous():   # its bytes are taken in one piece
        raise ValueError("ws is not contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _dense_bank(bank: Experts, H: int, device):
    bf = (torch.bfloat16,)
    wg, wu, wd = bank.w_gate, bank.w_up, bank.w_down
    if wg.dim() != 3 or bank.dt not in (None, BF16):
        raise ValueError("bank: bf16 weights [1][I][H] and [1][H][I]")
    I = wg.shape[1]
    if I > _MOST:
        raise ValueError(f"bank: I={I} is above {_MOST}")
    _tensor(device, "w_gate", wg, (1, I, H), bf)
    _tensor(device, "w_up", wu, (1, I, H), bf)
    _tensor(device, "w_down", wd, (1, H, I), bf)
    return ExpertsT(1, H, I, BF16, wg.data_ptr(), wu.data_ptr(), wd.data_ptr()), I


def ffn(x, bank: Experts, *, want_gu: bool = False, y_dtype=None, out=None, gu=None, ws=None, stream=None):
    """The dense gated FFN block (moe_ffn) with a bf16 bank of n = 1.  Returns
    y [T][H], or (y, gu) with want_gu: gu fp32 [T][2 I], what ffn_backward needs."""
    T, H, dev = _matrix("x", x)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return ffn(x, bank, want_gu=want_gu, y_dtype=y_dtype, out=out, gu=gu, ws=ws)
    st, I = _dense_bank(bank, H, dev)
    y_dtype = _out_dtype("out", out, y_dtype, torch.bfloat16)
    if y_dtype not in _FLOATS:
        raise TypeError(f"ffn: y {y_dtype}")
    _tensor(dev, "x", x, (T, H), (torch.bfloat16,))
    _tensor(dev, "out", out, (T, H), _FLOATS)
    _tensor(dev, "gu", gu, (T, 2 * I), (torch.float32,))
    if out is None:
        out = _empty(x, (T, H), y_dtype)
    if gu is None and want_gu:
        gu = _empty(x, (T, 2 * I), torch.float32)
    L = _lib or lib()
    wp, wn, ws = _scratch(ws, L.moe_ffn_workspace_size(T, H, I), x)
    _check(L.moe_ffn(x.data_ptr(), BF16, T, ctypes.byref(st), out.data_ptr(), _CODE[out.dtype], _ptr(gu), wp, wn,
                     _current(dev)))
    return (out, gu) if want_gu else out


def ffn_backward(dy, x, bank: Experts, gu=None, *, need=("dx", "dw_gate", "dw_up", "dw_down"), ws=None, stream=None):
    """Gradients of ffn (moe_ffn_backward): (dx [T][H], dw_gate, dw_up [1][I][H],
    dw_down [1][H][I]), None for those not in `need`.  gu: what ffn returned
    (None: computed again)."""
    T, H, dev = _matrix("x", x)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return ffn_backward(dy, x, bank, gu, need=need, ws=ws)
    st, I = _dense_bank(bank, H, dev)
    bf = (torch.bfloat16,)
    _tensor(dev, "x", x, (T, H), bf)
    _tensor(dev, "dy", dy, (T, H), bf)
    _tensor(dev, "gu", gu, (T, 2 * I), (torch.float32,))
    names = ("dx", "dw_gate", "dw_up", "dw_down")
    if not set(need) <= set(names):
        raise ValueError(f"need: {need}")
    likes = (x, bank.w_gate, bank.w_up, bank.w_down)
    o = tuple(torch.empty_like(t) if k in need else None for k, t in zip(names, likes))
    L = _lib or lib()
    wp, wn, ws = _scratch(ws, L.moe_ffn_backward_workspace_size(T, H, I, int(gu is not None)), x)
    _check(L.moe_ffn_backward(dy.data_ptr(), x.data_ptr(), BF16, T, ctypes.byref(st), _ptr(gu), *map(_ptr, o), wp, wn,
                              _current(dev)))
    return o


def _norm_params(T, H, dev, post_w, gate, gate_div, pre_w):
    """(rows of the gate, gate_div, weight dtype code) after the checks.  A
    gate_div of T or more is one gate for all tokens, whatever its size."""
    dtype = None
    for t in (post_w, gate, pre_w):
        if t is not None:
            if dtype is not None and t.dtype is not dtype:
                raise TypeError(f"post_w, gate and pre_w have different dtypes: {dtype}, {t.dtype}")
            dtype = t.dtype
    if dtype is None:
        return 0, 1, F32
    G = 0
    if gate is not None:
        if gate_div < 1:
            raise ValueError(f"gate_div={gate_div}")
        G = -(-T // gate_div)
        _tensor(dev, "gate", gate, (G, H), _FLOATS)
    _tensor(dev, "post_w", post_w, (H,), _FLOATS)
    _tensor(dev, "pre_w", pre_w, (H,), _FLOATS)
    return G, min(gate_div, _MOST), _CODE[dtype]


def norm(y, res=None, *, post_w=None, gate=None, gate_div: int = 1, res_scale: float = 1.0, pre_w=None,
         eps: float = 1e-6, r_dtype=None, x_dtype=None, want_r: bool = True, want_x: bool = True, r=None, x=None,
         stream=None):
    """The norm step between two blocks (moe_norm).  Returns (r, x); with
    x_dtype torch.int8 x is the pair (codes [T][H], scales [T]).  r has res's
    dtype, without res r_dtype (default: y's); x_dtype defaults to y's.  r, x:
    optional output tensors; r may be res itself."""
    T, H, dev = _matrix("y", y)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return norm(y, res, post_w=post_w, gate=gate, gate_div=gate_div, res_scale=res_scale, pre_w=pre_w, eps=eps,
                        r_dtype=r_dtype, x_dtype=x_dtype, want_r=want_r, want_x=want_x, r=r, x=x)
    _, gate_div, w_dt = _norm_params(T, H, dev, post_w, gate, gate_div, pre_w)
    r_dtype = _out_dtype("r", r, r_dtype, y.dtype) if res is None else _out_dtype("res", res, r_dtype, None)
    q, scale = x if isinstance(x, tuple) else (x, None)
    x_dtype = _out_dtype("x", q, x_dtype, y.dtype)
    if r_dtype not in _FLOATS or x_dtype not in _CODE:
        raise TypeError(f"norm: r {r_dtype}, x {x_dtype}")
    i8 = x_dtype == torch.int8
    if scale is not None and not i8:
        raise TypeError(f"norm: a scale for x of dtype {x_dtype}")
    _tensor(dev, "y", y, (T, H), _FLOATS)
    _tensor(dev, "res", res, (T, H), (r_dtype,))
    _tensor(dev, "r", r, (T, H), (r_dtype,))
    _tensor(dev, "x", q, (T, H), (x_dtype,))
    _tensor(dev, "x_scale", scale, (T,), (torch.float32,))
    if r is None and want_r:
        r = _empty(y if res is None else res, (T, H), r_dtype)
    if q is None and want_x:
        q = _empty(y, (T, H), x_dtype)
    if q is not None and i8 and scale is None:
        scale = _empty(y, (T,), torch.float32)
    L = _lib or lib()
    _check(L.moe_norm(y.data_ptr(), _CODE[y.dtype], _ptr(res), _CODE[r_dtype], T, H, _ptr(post_w), _ptr(gate), gate_div,
                      _ptr(pre_w), w_dt, res_scale, eps, _ptr(r), _ptr(q), _CODE[x_dtype], _ptr(scale), _current(dev)))
    return r, ((q, scale) if i8 and q is not None else q)


def norm_backward(dx, dr, y, r, *, post_w=None, gate=None, gate_div: int = 1, res_scale: float = 1.0, pre_w=None,
                  eps: float = 1e-6, need=("dy", "dres", "dpost_w", "dgate", "dpre_w"), ws=None, stream=None):
    """Gradients of norm (moe_norm_backward) as a dict with the keys dy (y's
    dtype), dres (r's), dpost_w, dgate and dpre_w (fp32); None for those that
    are not in `need` or have no input.  dx or dr may be None (zero), r with dx
    None, y without post_w and gate (dy then has dr's dtype, or r's)."""
    some = next((t for t in (y, r, dx, dr) if t is not None), None)
    if some is None:
        raise ValueError("norm_backward: no tensors")
    T, H, dev = _matrix("y, r, dx or dr", some)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return norm_backward(dx, dr, y, r, post_w=post_w, gate=gate, gate_div=gate_div, res_scale=res_scale,
                                 pre_w=pre_w, eps=eps, need=need, ws=ws)
    G, gate_div, w_dt = _norm_params(T, H, dev, post_w, gate, gate_div, pre_w)
    r_dtype = r.dtype if r is not None else dr.dtype if dr is not None else torch.float32
    y_dtype = y.dtype if y is not None else r_dtype
    _tensor(dev, "dx", dx, (T, H), _FLOATS)
    _tensor(dev, "dr", dr, (T, H), (r_dtype,))
    _tensor(dev, "y", y, (T, H), _FLOATS)
    _tensor(dev, "r", r, (T, H), _FLOATS)
    if r_dtype not in _FLOATS:
        raise TypeError(f"norm_backward: dr has dtype {r_dtype}")
    f32 = torch.float32
    what = {"dy": (some if y is None else y, (T, H), y_dtype), "dres": (some if r is None else r, (T, H), r_dtype),
            "dpost_w": (post_w, (H,), f32), "dgate": (gate, (G, H), f32), "dpre_w": (None if dx is None else pre_w, (H,), f32)}
    if not set(need) <= set(what):
        raise ValueError(f"need: {need}")
    o = {k: _empty(*v) if k in need and v[0] is not None else None for k, v in what.items()}
    L = _lib or lib()
    wp, wn, ws = _scratch(ws, L.moe_norm_backward_workspace_size(T, H, gate_div if gate is not None else 0), some)
    _check(L.moe_norm_backward(
        _ptr(dx), F32 if dx is None else _CODE[dx.dtype], _ptr(dr), _ptr(y), _CODE[y_dtype],
        _ptr(r), _CODE[r_dtype], T, H, _ptr(post_w), _ptr(gate), gate_div, _ptr(pre_w), w_dt,
        res_scale, eps, *map(_ptr, o.values()), wp, wn, _current(dev)))
    return o


def quant_i8(x, stream=None, out=None):
    """int8 codes [rows][cols], scales [rows] fp32 (moe_quant_i8)."""
    rows, cols, dev = _matrix("x", x)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return quant_i8(x, out=out)
    q, scale = out if out is not None else (None, None)
    _tensor(dev, "x", x, (rows, cols), _FLOATS)
    _tensor(dev, "q", q, (rows, cols), (torch.int8,))
    _tensor(dev, "scale", scale, (rows,), (torch.float32,))
    if out is None:
        q = _empty(x, (rows, cols), torch.int8)
        scale = _empty(x, (rows,), torch.float32)
    L = _lib or lib()
    _check(L.moe_quant_i8(x.data_ptr(), _CODE[x.dtype], rows, cols, q.data_ptr(), scale.data_ptr(), _current(dev)))
    return q, scale


def linear_i8(q, q_scale, w, w_scale, bias=None, *, out_dtype=None, out=None, ws=None, stream=None):
    """out [T][N] = (q w^T) * q_scale[:, None] * w_scale + bias (moe_linear_i8):
    q [T][K] and w [N][K] int8, q_scale [T], w_scale and bias [N] fp32."""
    T, K, dev = _matrix("q", q)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return linear_i8(q, q_scale, w, w_scale, bias, out_dtype=out_dtype, out=out, ws=ws)
    N = _matrix("w", w)[0]
    f32, i8 = (torch.float32,), (torch.int8,)
    out_dtype = _out_dtype("out", out, out_dtype, torch.bfloat16)
    if out_dtype not in _FLOATS:
        raise TypeError(f"linear_i8: out {out_dtype}")
    _tensor(dev, "q", q, (T, K), i8)
    _tensor(dev, "w", w, (N, K), i8)
    _tensor(dev, "q_scale", q_scale, (T,), f32)
    _tensor(dev, "w_scale", w_scale, (N,), f32)
    _tensor(dev, "bias", bias, (N,), f32)
    _tensor(dev, "out", out, (T, N), (out_dtype,))
    if out is None:
        out = _empty(q_scale, (T, N), out_dtype)
    L = _lib or lib()
    need = L.moe_linear_i8_workspace_size(T, K, N)
    wp, wn, ws = _scratch(ws, need, q) if need else (None, 0, None)
    _check(L.moe_linear_i8(q.data_ptr(), q_scale.data_ptr(), T, K, w.data_ptr(), w_scale.data_ptr(), _ptr(bias), N,
                           out.data_ptr(), _CODE[out_dtype], wp, wn, _current(dev)))
    return out
