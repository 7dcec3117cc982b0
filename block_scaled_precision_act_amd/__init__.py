"""Python binding of the gfx950 microscaling library (libmx_gfx950.so, C ABI in include/mx.h).

The functions below carry the C ABI's names and only marshal arguments: they take torch tensors
that already live on the GPU (torch is used for device memory and streams only), pass their
pointers, sizes and strides to the library and raise on a non-zero status.  Every step of the
computation runs in the library's HIP kernels; there is no fallback of any kind, and loading
fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmx_gfx950.so")

MX_OK, MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_STRIDE, MX_ERR_DEVICE, MX_ERR_LAUNCH = \
    0, -1, -2, -3, -4, -5, -6
MX_ERR_WORKSPACE = -7

_lib = None


class MxError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str | None = None):
        self.status = status
        msg = f"{fn} failed: status {status} ({status_str(status)})"
        super().__init__(msg if detail is None else f"{msg}: {detail}")


class MxCaps(ctypes.Structure):
    _fields_ = [("available", ctypes.c_int32), ("device", ctypes.c_int32),
                ("compute_units", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("arch", ctypes.c_char * 64), ("reason", ctypes.c_char * 128)]


_P, _I = ctypes.c_void_p, ctypes.c_int64
_SIGS = {
    "mx_capability": [ctypes.POINTER(MxCaps)],
    "mx_act_quant": [_P, _P, _P, _I, _I, _P],
    "mx_act_quant_strided_batched": [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P],
    "mx_act_quant_fp4": [_P, _P, _P, _I, _I, _P],
    "mx_act_quant_fp4_strided_batched": [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P],
}
for _n in ("fp8_fp4", "fp8_fp8", "fp4_fp4"):
    _SIGS[f"mx_gemm_{_n}"] = [_P, _P, _P, _P, _P, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_bias"] = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_strided_batched"] = [_P, _P, _P, _P, _P, _I, _I, _I, _I,
                                              _I, _I, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_bias_strided_batched"] = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                                   _I, _I, _I, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_bias_residual"] = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_bias_residual_strided_batched"] = [_P, _P, _P, _P, _P, _P, _P, _I, _I,
                                                            _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                                            _P]
    _SIGS[f"mx_gemm_{_n}_bias_gelu"] = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_bias_gelu_strided_batched"] = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                                        _I, _I, _I, _I, _I, _I, _P]
    _SIGS[f"mx_gemm_{_n}_splitk"] = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P]
_SIGS["mx_gemm_splitk_workspace_size"] = [_I, _I, _I]
_SIGS["mx_gemm_fp8_fp4_splitk_noalloc"] = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]
_U64, _C = ctypes.c_uint64, ctypes.c_int
_SIGS["mx_quant_e5m2"] = [_P, _P, _P, _I, _I, _C, _U64, _P]
_SIGS["mx_quant_e5m2_strided_batched"] = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _C, _U64, _P]
_SIGS["mx_quant_transpose_e4m3"] = [_P, _P, _P, _I, _I, _P]
_SIGS["mx_quant_transpose_e5m2"] = [_P, _P, _P, _I, _I, _C, _U64, _P]
_SIGS["mx_gemm_e5m2_e4m3"] = [_P, _P, _P, _P, _P, _I, _I, _I, _P]
_SIGS["mx_gemm_e5m2_e4m3_splitk"] = [_P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P]
_SIGS["mx_gemm_e5m2_e4m3_strided_batched"] = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                                              _I, _P]
for _n in ("fp8_fp4", "fp8_fp8", "fp4_fp4"):
    for _v in ("_quant", "_bias_gelu_quant"):
        _SIGS[f"mx_gemm_{_n}{_v}"] = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]
        _SIGS[f"mx_gemm_{_n}{_v}_strided_batched"] = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                                      _I, _I, _I, _I, _I, _I, _I, _P]
# Attention operators (include/mx_attention.h): an argument struct and the stream.
for _n in ("mx_qk_norm_rope", "mx_qk_norm_rope_backward", "mx_kv_append_fp4", "mx_attn_fp4"):
    _SIGS[_n] = [ctypes.c_char_p, _P]
_SIGS["mx_qk_norm_rope_backward_workspace_size"] = [_I, _I, _I, _I]
_SIGS["mx_attn_fp4_workspace_size"] = [_I, _I, _I, _I, _I]
_INT64_RESULTS = ("mx_gemm_splitk_workspace_size", "mx_qk_norm_rope_backward_workspace_size",
                  "mx_attn_fp4_workspace_size")


def load(path: str | None = None) -> ctypes.CDLL:
    """Loads the built library (raises when it is missing: there is no other implementation)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -m block_scaled_precision_act_amd.build`")
    lib = ctypes.CDLL(p)
    for name, argtypes in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    lib.mx_status_str.argtypes = [ctypes.c_int]
    lib.mx_status_str.restype = ctypes.c_char_p
    for name in _INT64_RESULTS:
        getattr(lib, name).restype = ctypes.c_int64
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().mx_status_str(status).decode()


def mx_capability() -> dict:
    caps = MxCaps()
    st = load().mx_capability(ctypes.byref(caps))
    return {"status": st, "available": bool(caps.available), "device": caps.device,
            "compute_units": caps.compute_units, "arch": caps.arch.decode(),
            "reason": caps.reason.decode()}


_RAW_STREAM = []


def _stream(stream):
    """The hipStream_t to launch on: `stream` (a torch stream or a raw handle), else torch's
    current stream on the current device (through torch's raw-handle getter where it exists,
    which skips building a stream object: 0.06 instead of 2.7 us per call)."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if not _RAW_STREAM:
        import torch
        _RAW_STREAM.append(getattr(torch._C, "_cuda_getCurrentRawStream", None))
    raw = _RAW_STREAM[0]
    if raw is not None:
        return raw(_current_device())
    import torch
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


_DT = {}


def _dtypes():
    if not _DT:
        import torch
        _DT.update(u8=torch.uint8, bf16=torch.bfloat16, tensor=torch.Tensor,
                   current=torch.cuda.current_device)
    return _DT


def _current_device() -> int:
    """The current GPU's index, or -1 when no GPU is visible (every tensor is then refused)."""
    try:
        return _dtypes()["current"]()
    except Exception:
        return -1


def _need(fn: str, t, what: str, dtype: str, rows: int, cols: int, batch: int | None = None,
          output: bool = False, dev: int | None = None):
    """Checks that tensor `t` can be passed to the library as `what`: a tensor on the current GPU
    (index `dev`, queried once per call by the caller when given) of dtype `dtype` ("u8" or
    "bf16") shaped [rows, cols], or [batch, rows, cols] in a batched call (an input may also be a
    single [rows, cols] matrix, broadcast to every batch), whose rows are contiguous (column
    stride 1, row stride cols) as the library addresses them.  The library sees only pointers, so
    a host tensor or a buffer smaller than this would be read or written out of bounds on the
    GPU; such arguments raise here instead."""
    dt = _DT or _dtypes()
    if not isinstance(t, dt["tensor"]):
        raise TypeError(f"{fn}: {what} must be a torch tensor, got {type(t).__name__}")
    d = t.get_device()
    if d < 0 or d != (_current_device() if dev is None else dev):
        raise MxError(fn, MX_ERR_DEVICE, f"{what} is on {t.device}, not the current GPU")
    if t.dtype is not dt[dtype]:
        raise TypeError(f"{fn}: {what} must be {dt[dtype]}, got {t.dtype}")
    sh = t.shape
    nd = len(sh)
    if batch is None:
        ok = nd == 2
    elif output:
        ok = nd == 3 and sh[0] == batch
    else:
        ok = nd == 2 or (nd == 3 and sh[0] == batch)
    if not ok or sh[-2] != rows or sh[-1] != cols:
        lead = "" if batch is None else f"{batch}, "
        raise MxError(fn, MX_ERR_SHAPE, f"{what} has shape {tuple(sh)}, expected "
                                        f"[{lead}{rows}, {cols}]")
    if t.is_contiguous():          # rows of cols elements, one after another
        return
    st = t.stride()
    if rows and cols and (cols > 1 and st[-1] != 1 or rows > 1 and st[-2] != cols or
                          nd == 3 and st[0] < 0):
        raise MxError(fn, MX_ERR_STRIDE, f"{what} rows are not contiguous (strides {st})")


def _need_bias(fn: str, bias, N: int, batch: int | None, dev: int | None = None):
    """bias: bf16 [N], or [batch, N] in a batched call (a [N] bias is shared by every batch)."""
    if bias is None:
        return
    dt = _DT or _dtypes()
    if not isinstance(bias, dt["tensor"]):
        raise TypeError(f"{fn}: bias must be a torch tensor, got {type(bias).__name__}")
    d = bias.get_device()
    if d < 0 or d != (_current_device() if dev is None else dev):
        raise MxError(fn, MX_ERR_DEVICE, f"bias is on {bias.device}, not the current GPU")
    if bias.dtype is not dt["bf16"]:
        raise TypeError(f"{fn}: bias must be {dt['bf16']}, got {bias.dtype}")
    sh = bias.shape
    if not (len(sh) == 1 or (batch is not None and len(sh) == 2 and sh[0] == batch)) or \
            sh[-1] != N:
        raise MxError(fn, MX_ERR_SHAPE, f"bias has shape {tuple(sh)}, expected [{N}]" +
                      ("" if batch is None else f" or [{batch}, {N}]"))
    if N > 1 and bias.stride(-1) != 1 or len(sh) == 2 and bias.stride(0) < 0:
        raise MxError(fn, MX_ERR_STRIDE, f"bias elements are not contiguous ({bias.stride()})")


def _need_workspace(fn: str, ws):
    import torch
    if ws is None:
        return
    if not isinstance(ws, torch.Tensor) or ws.device.type != "cuda" or \
            ws.device.index != torch.cuda.current_device():
        raise MxError(fn, MX_ERR_DEVICE, "the workspace must be a tensor on the current GPU")
    if not ws.is_contiguous():
        raise MxError(fn, MX_ERR_STRIDE, "the workspace must be contiguous")


# Operand shapes per GEMM kind: (A columns, B rows, B columns, B scale rows) for M, N, K.
def _operand_shapes(kind: str, N: int, K: int):
    a_cols = K // 2 if kind == "fp4_fp4" else K
    b_cols = K if kind in ("fp8_fp8", "e5m2_e4m3") else K // 2
    bs_rows = _cdiv(N, 32) if kind == "fp8_fp8" else N
    return a_cols, b_cols, bs_rows


def _need_operands(fn: str, kind: str, a, a_s, b, b_s, M: int, N: int, K: int,
                   batch: int | None, dev: int | None = None):
    a_cols, b_cols, bs_rows = _operand_shapes(kind, N, K)
    kb = _cdiv(K, 32)
    _need(fn, a, "a", "u8", M, a_cols, batch, dev=dev)
    _need(fn, a_s, "a_s", "u8", M, kb, batch, dev=dev)
    _need(fn, b, "b", "u8", N, b_cols, batch, dev=dev)
    _need(fn, b_s, "b_s", "u8", bs_rows, kb, batch, dev=dev)


def _k_of(kind: str, a) -> int:
    return a.shape[-1] * (2 if kind == "fp4_fp4" else 1)


def _check(fn: str, st: int):
    if st != MX_OK:
        raise MxError(fn, st)


def mx_act_quant(x, q, s, stream=None):
    """x: bf16 [M, K] (cuda); q: uint8 [M, K]; s: uint8 [M, K/32] (written)."""
    M, K = x.shape[-2], x.shape[-1]
    dev = _current_device()
    _need("mx_act_quant", x, "x", "bf16", M, K, dev=dev)
    _need("mx_act_quant", q, "q", "u8", M, K, dev=dev)
    _need("mx_act_quant", s, "s", "u8", M, _cdiv(K, 32), dev=dev)
    _check("mx_act_quant", load().mx_act_quant(_ptr(x), _ptr(q), _ptr(s), M, K, _stream(stream)))


def mx_act_quant_strided_batched(x, q, s, stream=None):
    """x: bf16 [B, M, K]; q: uint8 [B, M, K]; s: uint8 [B, M, K/32]; batch strides from the
    tensors (a stride-0 x broadcasts)."""
    B, M, K = x.shape
    fn = "mx_act_quant_strided_batched"
    dev = _current_device()
    _need(fn, x, "x", "bf16", M, K, B, output=True, dev=dev)
    _need(fn, q, "q", "u8", M, K, B, output=True, dev=dev)
    _need(fn, s, "s", "u8", M, _cdiv(K, 32), B, output=True, dev=dev)
    _check("mx_act_quant_strided_batched",
           load().mx_act_quant_strided_batched(_ptr(x), _ptr(q), _ptr(s), M, K, B,
                                               x.stride(0), q.stride(0), s.stride(0),
                                               _stream(stream)))


def mx_act_quant_fp4(x, q, s, stream=None):
    """x: bf16 [M, K] (cuda); q: uint8 [M, K/2] packed E2M1; s: uint8 [M, K/32] (written)."""
    M, K = x.shape[-2], x.shape[-1]
    dev = _current_device()
    _need("mx_act_quant_fp4", x, "x", "bf16", M, K, dev=dev)
    _need("mx_act_quant_fp4", q, "q", "u8", M, K // 2, dev=dev)
    _need("mx_act_quant_fp4", s, "s", "u8", M, _cdiv(K, 32), dev=dev)
    _check("mx_act_quant_fp4",
           load().mx_act_quant_fp4(_ptr(x), _ptr(q), _ptr(s), M, K, _stream(stream)))


def mx_act_quant_fp4_strided_batched(x, q, s, stream=None):
    """x: bf16 [B, M, K]; q: uint8 [B, M, K/2]; s: uint8 [B, M, K/32]; strides from the tensors."""
    B, M, K = x.shape
    fn = "mx_act_quant_fp4_strided_batched"
    dev = _current_device()
    _need(fn, x, "x", "bf16", M, K, B, output=True, dev=dev)
    _need(fn, q, "q", "u8", M, K // 2, B, output=True, dev=dev)
    _need(fn, s, "s", "u8", M, _cdiv(K, 32), B, output=True, dev=dev)
    _check("mx_act_quant_fp4_strided_batched",
           load().mx_act_quant_fp4_strided_batched(_ptr(x), _ptr(q), _ptr(s), M, K, B,
                                                   x.stride(0), q.stride(0), s.stride(0),
                                                   _stream(stream)))


def _gemm(kind: str, a, a_s, b, b_s, c, bias=None, K=None, stream=None):
    M, N = c.shape[-2], c.shape[-1]
    if K is None:
        K = _k_of(kind, a)
    batch = c.shape[0] if c.dim() == 3 else None
    fn = f"mx_gemm_{kind}"
    dev = _current_device()
    _need(fn, c, "c", "bf16", M, N, batch, output=True, dev=dev)
    _need_operands(fn, kind, a, a_s, b, b_s, M, N, K, batch, dev=dev)
    _need_bias(fn, bias, N, batch, dev=dev)
    lib = load()
    st = _stream(stream)
    if c.dim() == 2:
        if bias is None:
            r = getattr(lib, f"mx_gemm_{kind}")(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(c),
                                                M, N, K, st)
        else:
            r = getattr(lib, f"mx_gemm_{kind}_bias")(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s),
                                                     _ptr(bias), _ptr(c), M, N, K, st)
        name = f"mx_gemm_{kind}" + ("" if bias is None else "_bias")
    else:
        B = c.shape[0]
        strides = [t.stride(0) if t.dim() == 3 else 0 for t in (a, a_s, b, b_s)]
        if bias is None:
            r = getattr(lib, f"mx_gemm_{kind}_strided_batched")(
                _ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(c), M, N, K, B, *strides,
                c.stride(0), st)
            name = f"mx_gemm_{kind}_strided_batched"
        else:
            sbias = bias.stride(0) if bias.dim() == 2 else 0
            r = getattr(lib, f"mx_gemm_{kind}_bias_strided_batched")(
                _ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(bias), _ptr(c), M, N, K, B,
                *strides, sbias, c.stride(0), st)
            name = f"mx_gemm_{kind}_bias_strided_batched"
    _check(name, r)


def mx_gemm_fp8_fp4(a, a_s, b, b_s, c, bias=None, stream=None):
    """a: E4M3 [(B,) M, K]; a_s: [(B,) M, K/32]; b: packed E2M1 [(B,) N, K/2]; b_s: [(B,) N, K/32];
    c: bf16 [(B,) M, N]; bias: bf16 [(B,) N] or None.  A 2-D operand of a batched call is
    broadcast (stride 0)."""
    _gemm("fp8_fp4", a, a_s, b, b_s, c, bias, K=a.shape[-1], stream=stream)


def mx_gemm_fp8_fp8(a, a_s, b, b_s, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4 with b: E4M3 [(B,) N, K] and b_s: [(B,) ceil(N/32), K/32]."""
    _gemm("fp8_fp8", a, a_s, b, b_s, c, bias, K=a.shape[-1], stream=stream)


def mx_gemm_fp4_fp4(a, a_s, b, b_s, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4 with a: packed E2M1 [(B,) M, K/2]."""
    _gemm("fp4_fp4", a, a_s, b, b_s, c, bias, K=2 * a.shape[-1], stream=stream)


def _gemm_quant(kind: str, a, a_s, b, b_s, q, q_s, bias=None, stream=None, gelu=False):
    fp4 = kind == "fp4_fp4"
    M, K = q.shape[-2], a.shape[-1] * (2 if fp4 else 1)
    N = q.shape[-1] * (2 if fp4 else 1)
    v = "_bias_gelu_quant" if gelu else "_quant"
    batch = q.shape[0] if q.dim() == 3 else None
    fn = f"mx_gemm_{kind}{v}"
    dev = _current_device()
    _need(fn, q, "q", "u8", M, q.shape[-1], batch, output=True, dev=dev)
    _need(fn, q_s, "q_s", "u8", M, _cdiv(N, 32), batch, output=True, dev=dev)
    _need_operands(fn, kind, a, a_s, b, b_s, M, N, K, batch, dev=dev)
    _need_bias(fn, bias, N, batch, dev=dev)
    lib = load()
    st = _stream(stream)
    if q.dim() == 2:
        name = f"mx_gemm_{kind}{v}"
        r = getattr(lib, name)(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(bias), _ptr(q),
                               _ptr(q_s), M, N, K, st)
    else:
        B = q.shape[0]
        strides = [t.stride(0) if t.dim() == 3 else 0 for t in (a, a_s, b, b_s)]
        sbias = bias.stride(0) if (bias is not None and bias.dim() == 2) else 0
        name = f"mx_gemm_{kind}{v}_strided_batched"
        r = getattr(lib, name)(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(bias), _ptr(q),
                               _ptr(q_s), M, N, K, B, *strides, sbias, q.stride(0),
                               q_s.stride(0), st)
    _check(name, r)


def mx_gemm_fp8_fp4_quant(a, a_s, b, b_s, q, q_s, bias=None, stream=None):
    """As mx_gemm_fp8_fp4, but the bf16 output is written as the next layer's activation operand:
    q: E4M3 [(B,) M, N] and q_s: E8M0 [(B,) M, N/32] (N % 32 == 0)."""
    _gemm_quant("fp8_fp4", a, a_s, b, b_s, q, q_s, bias, stream)


def mx_gemm_fp8_fp8_quant(a, a_s, b, b_s, q, q_s, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_quant with b: E4M3 [(B,) N, K] and b_s: [(B,) ceil(N/32), K/32]."""
    _gemm_quant("fp8_fp8", a, a_s, b, b_s, q, q_s, bias, stream)


def mx_gemm_fp4_fp4_quant(a, a_s, b, b_s, q, q_s, bias=None, stream=None):
    """A4W4 GEMM whose bf16 output is written as the next A4W4 layer's operand: q packed E2M1
    [(B,) M, N/2] and q_s E8M0 [(B,) M, N/32] (N % 32 == 0)."""
    _gemm_quant("fp4_fp4", a, a_s, b, b_s, q, q_s, bias, stream)


def mx_gemm_fp8_fp4_bias_gelu_quant(a, a_s, b, b_s, q, q_s, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_quant with GELU applied before the bf16 rounding that is quantized."""
    _gemm_quant("fp8_fp4", a, a_s, b, b_s, q, q_s, bias, stream, gelu=True)


def mx_gemm_fp8_fp8_bias_gelu_quant(a, a_s, b, b_s, q, q_s, bias=None, stream=None):
    """As mx_gemm_fp8_fp8_quant with GELU applied before the bf16 rounding that is quantized."""
    _gemm_quant("fp8_fp8", a, a_s, b, b_s, q, q_s, bias, stream, gelu=True)


def mx_gemm_fp4_fp4_bias_gelu_quant(a, a_s, b, b_s, q, q_s, bias=None, stream=None):
    """As mx_gemm_fp4_fp4_quant with GELU applied before the bf16 rounding that is quantized."""
    _gemm_quant("fp4_fp4", a, a_s, b, b_s, q, q_s, bias, stream, gelu=True)


def _gemm_epilogue(kind: str, epi: str, a, a_s, b, b_s, c, bias=None, residual=None,
                   stream=None):
    M, N = c.shape[-2], c.shape[-1]
    K = _k_of(kind, a)
    batch = c.shape[0] if c.dim() == 3 else None
    fn = f"mx_gemm_{kind}_bias_{epi}"
    dev = _current_device()
    _need(fn, c, "c", "bf16", M, N, batch, output=True, dev=dev)
    _need_operands(fn, kind, a, a_s, b, b_s, M, N, K, batch, dev=dev)
    _need_bias(fn, bias, N, batch, dev=dev)
    if epi == "residual":
        _need(fn, residual, "residual", "bf16", M, N, batch, dev=dev)
    lib = load()
    st = _stream(stream)
    res = [_ptr(residual)] if epi == "residual" else []
    if c.dim() == 2:
        name = f"mx_gemm_{kind}_bias_{epi}"
        r = getattr(lib, name)(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(bias), *res, _ptr(c),
                               M, N, K, st)
    else:
        B = c.shape[0]
        strides = [t.stride(0) if t.dim() == 3 else 0 for t in (a, a_s, b, b_s)]
        sbias = bias.stride(0) if (bias is not None and bias.dim() == 2) else 0
        sres = [residual.stride(0) if residual.dim() == 3 else 0] if epi == "residual" else []
        name = f"mx_gemm_{kind}_bias_{epi}_strided_batched"
        r = getattr(lib, name)(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(bias), *res, _ptr(c),
                               M, N, K, B, *strides, sbias, *sres, c.stride(0), st)
    _check(name, r)


def mx_gemm_fp8_fp4_bias_residual(a, a_s, b, b_s, residual, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4 with a bf16 residual [(B,) M, N] added before the one bf16 rounding
    (residual may be c itself); bias optional."""
    _gemm_epilogue("fp8_fp4", "residual", a, a_s, b, b_s, c, bias, residual, stream)


def mx_gemm_fp8_fp8_bias_residual(a, a_s, b, b_s, residual, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_bias_residual for FP8 weights."""
    _gemm_epilogue("fp8_fp8", "residual", a, a_s, b, b_s, c, bias, residual, stream)


def mx_gemm_fp4_fp4_bias_residual(a, a_s, b, b_s, residual, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_bias_residual for MXFP4 activations."""
    _gemm_epilogue("fp4_fp4", "residual", a, a_s, b, b_s, c, bias, residual, stream)


def mx_gemm_fp8_fp4_bias_gelu(a, a_s, b, b_s, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4 with GELU (x * Phi(x)) applied to sum + bias before the one bf16
    rounding; bias optional."""
    _gemm_epilogue("fp8_fp4", "gelu", a, a_s, b, b_s, c, bias, None, stream)


def mx_gemm_fp8_fp8_bias_gelu(a, a_s, b, b_s, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_bias_gelu for FP8 weights."""
    _gemm_epilogue("fp8_fp8", "gelu", a, a_s, b, b_s, c, bias, None, stream)


def mx_gemm_fp4_fp4_bias_gelu(a, a_s, b, b_s, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_bias_gelu for MXFP4 activations."""
    _gemm_epilogue("fp4_fp4", "gelu", a, a_s, b, b_s, c, bias, None, stream)


def mx_gemm_splitk_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace the _splitk entry points need for an M x N x K problem (0: not split)."""
    return int(load().mx_gemm_splitk_workspace_size(M, N, K))


def _gemm_splitk(kind: str, a, a_s, b, b_s, c, workspace, bias=None, stream=None):
    M, N = c.shape
    K = _k_of(kind, a)
    fn = f"mx_gemm_{kind}_splitk"
    dev = _current_device()
    _need(fn, c, "c", "bf16", M, N, dev=dev)
    _need_operands(fn, kind, a, a_s, b, b_s, M, N, K, None, dev=dev)
    _need_bias(fn, bias, N, None, dev=dev)
    _need_workspace(fn, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    name = f"mx_gemm_{kind}_splitk"
    _check(name, getattr(load(), name)(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(bias),
                                       _ptr(c), M, N, K, _ptr(workspace), ws_bytes,
                                       _stream(stream)))


def mx_gemm_fp8_fp4_splitk(a, a_s, b, b_s, c, workspace, bias=None, stream=None):
    """As mx_gemm_fp8_fp4 (single problem) with K split across workgroups when the shape has few
    output tiles; workspace: a zero-filled device buffer of mx_gemm_splitk_workspace_size bytes
    (256-byte aligned; left reusable), or None for shapes that are not split."""
    _gemm_splitk("fp8_fp4", a, a_s, b, b_s, c, workspace, bias, stream)


def mx_gemm_fp8_fp4_splitk_noalloc(a, a_s, b, b_s, c, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_splitk without a workspace: the library's fixed device array holds the
    partial tiles (calls on one GPU must not overlap)."""
    M, N = c.shape
    K = _k_of("fp8_fp4", a)
    fn = "mx_gemm_fp8_fp4_splitk_noalloc"
    dev = _current_device()
    _need(fn, c, "c", "bf16", M, N, dev=dev)
    _need_operands(fn, "fp8_fp4", a, a_s, b, b_s, M, N, K, None, dev=dev)
    _need_bias(fn, bias, N, None, dev=dev)
    _check(fn, load().mx_gemm_fp8_fp4_splitk_noalloc(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s),
                                                     _ptr(bias), _ptr(c), M, N, K,
                                                     _stream(stream)))


def mx_gemm_fp8_fp8_splitk(a, a_s, b, b_s, c, workspace, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_splitk for FP8 weights."""
    _gemm_splitk("fp8_fp8", a, a_s, b, b_s, c, workspace, bias, stream)


def mx_gemm_fp4_fp4_splitk(a, a_s, b, b_s, c, workspace, bias=None, stream=None):
    """As mx_gemm_fp8_fp4_splitk for MXFP4 activations."""
    _gemm_splitk("fp4_fp4", a, a_s, b, b_s, c, workspace, bias, stream)


def mx_quant_e5m2(x, q, s, seed=None, stream=None):
    """Gradients x: bf16 [(B,) M, K] -> q: E5M2 [(B,) M, K], s: E8M0 [(B,) M, K/32]; round to
    nearest even (seed None) or stochastically from Philox4x64-10 under `seed`."""
    st, sd = (0, 0) if seed is None else (1, int(seed))
    M, K = x.shape[-2], x.shape[-1]
    batch = x.shape[0] if x.dim() == 3 else None
    fn = "mx_quant_e5m2"
    dev = _current_device()
    _need(fn, x, "x", "bf16", M, K, batch, output=True, dev=dev)
    _need(fn, q, "q", "u8", M, K, batch, output=True, dev=dev)
    _need(fn, s, "s", "u8", M, _cdiv(K, 32), batch, output=True, dev=dev)
    if x.dim() == 2:
        _check("mx_quant_e5m2", load().mx_quant_e5m2(_ptr(x), _ptr(q), _ptr(s), M, K, st, sd,
                                                     _stream(stream)))
    else:
        _check("mx_quant_e5m2_strided_batched",
               load().mx_quant_e5m2_strided_batched(_ptr(x), _ptr(q), _ptr(s), M, K, x.shape[0],
                                                    x.stride(0), q.stride(0), s.stride(0), st, sd,
                                                    _stream(stream)))


def mx_quant_transpose_e4m3(x, q, s, stream=None):
    """x: bf16 [R, C] -> q: E4M3 [C, R], s: E8M0 [C, R/32] (act_quant of x^T)."""
    R, C = x.shape
    fn = "mx_quant_transpose_e4m3"
    dev = _current_device()
    _need(fn, x, "x", "bf16", R, C, dev=dev)
    _need(fn, q, "q", "u8", C, R, dev=dev)
    _need(fn, s, "s", "u8", C, _cdiv(R, 32), dev=dev)
    _check("mx_quant_transpose_e4m3",
           load().mx_quant_transpose_e4m3(_ptr(x), _ptr(q), _ptr(s), R, C, _stream(stream)))


def mx_quant_transpose_e5m2(x, q, s, seed=None, stream=None):
    """x: bf16 [R, C] -> q: E5M2 [C, R], s: E8M0 [C, R/32] (mx_quant_e5m2 of x^T)."""
    R, C = x.shape
    fn = "mx_quant_transpose_e5m2"
    dev = _current_device()
    _need(fn, x, "x", "bf16", R, C, dev=dev)
    _need(fn, q, "q", "u8", C, R, dev=dev)
    _need(fn, s, "s", "u8", C, _cdiv(R, 32), dev=dev)
    st, sd = (0, 0) if seed is None else (1, int(seed))
    _check("mx_quant_transpose_e5m2",
           load().mx_quant_transpose_e5m2(_ptr(x), _ptr(q), _ptr(s), R, C, st, sd,
                                          _stream(stream)))


def mx_gemm_e5m2_e4m3(a, a_s, b, b_s, c, stream=None):
    """a: E5M2 [(B,) M, K] + a_s [(B,) M, K/32]; b: E4M3 [(B,) N, K] + b_s [(B,) N, K/32] (per-row
    scales); c: bf16 [(B,) M, N] = a b^T."""
    M, N, K = c.shape[-2], c.shape[-1], a.shape[-1]
    batch = c.shape[0] if c.dim() == 3 else None
    fn = "mx_gemm_e5m2_e4m3"
    dev = _current_device()
    _need(fn, c, "c", "bf16", M, N, batch, output=True, dev=dev)
    _need_operands(fn, "e5m2_e4m3", a, a_s, b, b_s, M, N, K, batch, dev=dev)
    lib = load()
    if c.dim() == 2:
        _check("mx_gemm_e5m2_e4m3", lib.mx_gemm_e5m2_e4m3(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s),
                                                          _ptr(c), M, N, K, _stream(stream)))
    else:
        strides = [t.stride(0) if t.dim() == 3 else 0 for t in (a, a_s, b, b_s)]
        _check("mx_gemm_e5m2_e4m3_strided_batched",
               lib.mx_gemm_e5m2_e4m3_strided_batched(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s),
                                                     _ptr(c), M, N, K, c.shape[0], *strides,
                                                     c.stride(0), _stream(stream)))


def mx_gemm_e5m2_e4m3_splitk(a, a_s, b, b_s, c, workspace, stream=None):
    """As mx_gemm_e5m2_e4m3 (single problem) with K split across workgroups for shapes with few
    output tiles; workspace as for mx_gemm_fp8_fp4_splitk (None where the shape is not split)."""
    M, N, K = c.shape[0], c.shape[1], a.shape[-1]
    fn = "mx_gemm_e5m2_e4m3_splitk"
    dev = _current_device()
    _need(fn, c, "c", "bf16", M, N, dev=dev)
    _need_operands(fn, "e5m2_e4m3", a, a_s, b, b_s, M, N, K, None, dev=dev)
    _need_workspace(fn, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("mx_gemm_e5m2_e4m3_splitk",
           load().mx_gemm_e5m2_e4m3_splitk(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), _ptr(c), M, N,
                                           K, _ptr(workspace), ws_bytes, _stream(stream)))


# The attention operators (include/mx_attention.h) are in attention.py, imported when first used.
_ATTENTION = ("MxKvCacheFp4", "mx_attn_fp4", "mx_attn_fp4_workspace_size", "mx_kv_append_fp4",
              "mx_qk_norm_rope", "mx_qk_norm_rope_backward",
              "mx_qk_norm_rope_backward_workspace_size")


def __getattr__(name):
    if name not in _ATTENTION:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import attention
    globals().update({n: getattr(attention, n) for n in _ATTENTION})
    return globals()[name]
