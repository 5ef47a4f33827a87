"""ctypes binding of libmoedecode (include/moedecode.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels. Tensors are torch CUDA tensors (device memory on the current device);
the stream is torch's current stream unless one is given. There is no CPU
fallback -- if the shared library is missing or fails to load, importing the
functions raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoedecode.so")

(MOED_OK, MOED_ERR_NULL, MOED_ERR_SHAPE, MOED_ERR_DTYPE, MOED_ERR_WORKSPACE, MOED_ERR_ALIGN, MOED_ERR_HIP,
 MOED_ERR_SCALE, MOED_ERR_TUNING) = range(9)
MOED_BF16, MOED_F32 = 0, 1
MOED_ROWS_BF16, MOED_ROWS_F32, MOED_ROWS_MXFP8, MOED_ROWS_MXFP8_FAST = 0, 1, 2, 4

EXPORTS = ("moed_workspace_bytes", "moe_decode", "moe_decode_gate_up", "moe_decode_down", "moe_route",
           "moed_selftest_decode", "moed_bench_read", "moed_bench_copy", "moed_status_string",
           "moed_last_hip_error", "moed_tuning_init", "moe_decode_tuned", "moe_decode_gate_up_tuned",
           "moe_decode_down_tuned", "moe_decode_noalloc", "moed_bench_read_cfg", "moe_norm",
           "moe_group_workspace_bytes", "moe_group", "moe_grouped_workspace_bytes", "moe_grouped_gate_up",
           "moe_grouped_matmul", "moe_combine", "moe_prefill_workspace_bytes", "moe_prefill")


class MoedTuning(ctypes.Structure):
    """moed_tuning of the header: a launch-shape choice handed to one call."""
    _fields_ = [("words", ctypes.c_int32 * 48)]


class MoedError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.moed_status_string(status).decode()
        if status == MOED_ERR_HIP:
            msg += f" (hipError {lib.moed_last_hip_error()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libmoedecode.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} not built: run __graft_entry__.build() "
                              "(or python -m output_centric_expert_amd.build)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.moed_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.moed_workspace_bytes.restype = Z
        lib.moe_decode.argtypes = [P] * 9 + [I, P] + [I] * 7 + [P, Z, P]
        lib.moe_decode.restype = I
        lib.moe_decode_gate_up.argtypes = [P] * 6 + [I, P] + [I] * 6 + [P]
        lib.moe_decode_gate_up.restype = I
        lib.moe_decode_down.argtypes = [P, I, P, P, P, P, I, P, I] + [I] * 5 + [P, Z, P]
        lib.moe_decode_down.restype = I
        lib.moe_decode_noalloc.argtypes = [P] * 9 + [I, P] + [I] * 7 + [P]
        lib.moe_decode_noalloc.restype = I
        TP = ctypes.POINTER(MoedTuning)
        lib.moed_tuning_init.argtypes = [TP, ctypes.c_char_p]
        lib.moed_tuning_init.restype = I
        lib.moe_decode_tuned.argtypes = lib.moe_decode.argtypes + [TP]
        lib.moe_decode_tuned.restype = I
        lib.moe_decode_gate_up_tuned.argtypes = lib.moe_decode_gate_up.argtypes + [TP]
        lib.moe_decode_gate_up_tuned.restype = I
        lib.moe_decode_down_tuned.argtypes = lib.moe_decode_down.argtypes + [TP]
        lib.moe_decode_down_tuned.restype = I
        lib.moe_route.argtypes = [P, I, I, I, I, ctypes.c_float, P, P, P]
        lib.moe_route.restype = I
        lib.moe_norm.argtypes = [P, I, P, I, P, I, ctypes.c_float, P, P, I, P, P, I, I, P]
        lib.moe_norm.restype = I
        lib.moe_group_workspace_bytes.argtypes = [I, I, I]
        lib.moe_group_workspace_bytes.restype = Z
        lib.moe_group.argtypes = [P, I, I, I, P, P, P, P, Z, P]
        lib.moe_group.restype = I
        lib.moe_grouped_workspace_bytes.argtypes = [I] * 6
        lib.moe_grouped_workspace_bytes.restype = Z
        lib.moe_grouped_gate_up.argtypes = [P, P, I, I, P, I] + [P] * 5 + [I, P, P, I] + [I] * 4 + [P, Z, P]
        lib.moe_grouped_gate_up.restype = I
        lib.moe_grouped_matmul.argtypes = [P, P, I, I, P, I] + [P] * 3 + [I, P, I] + [I] * 4 + [P, Z, P]
        lib.moe_grouped_matmul.restype = I
        lib.moe_combine.argtypes = [P, I, I, P, P, P, I, I, I, I, P]
        lib.moe_combine.restype = I
        lib.moe_prefill_workspace_bytes.argtypes = [I] * 7
        lib.moe_prefill_workspace_bytes.restype = Z
        lib.moe_prefill.argtypes = [P, P, I] + [P] * 8 + [I, P, I] + [I] * 5 + [P, Z, P]
        lib.moe_prefill.restype = I
        lib.moed_selftest_decode.argtypes = [P, P, P, I, I, P]
        lib.moed_selftest_decode.restype = I
        lib.moed_bench_read.argtypes = [P, Z, P, Z, P]
        lib.moed_bench_read.restype = I
        lib.moed_bench_read_cfg.argtypes = [P, Z, P, Z, I, I, I, P]
        lib.moed_bench_read_cfg.restype = I
        lib.moed_bench_copy.argtypes = [P, P, Z, P]
        lib.moed_bench_copy.restype = I
        lib.moed_status_string.argtypes = [I]
        lib.moed_status_string.restype = ctypes.c_char_p
        lib.moed_last_hip_error.argtypes = []
        lib.moed_last_hip_error.restype = I
        _lib = lib
    return _lib


_DT = {torch.bfloat16: MOED_BF16, torch.float32: MOED_F32}


def _ptr(t: torch.Tensor | None, name: str, dtype=None, shape=None, cuda=True):
    if t is None:
        return None
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else ctypes.c_void_p(0)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(st: int, where: str):
    if st != MOED_OK:
        raise MoedError(st, where)


def moed_tuning_init(spec: str | None) -> MoedTuning:
    """A moed_tuning filled from the built-in table and `spec` ("key=value,...")."""
    t = MoedTuning()
    _check(load().moed_tuning_init(ctypes.byref(t), spec.encode() if spec else None), "moed_tuning_init")
    return t


_default = threading.local()


def set_default_tuning(spec: str | None):
    """Later calls made by this Python thread without a tuning argument pass a moed_tuning
    filled from `spec` (None: the built-in table). A convenience of the binding for tests and
    sweeps; the library itself keeps no state between calls."""
    _default.tuning = moed_tuning_init(spec) if spec else None


@contextlib.contextmanager
def tuned(spec: str | None):
    """set_default_tuning(spec) for the calls inside the block."""
    prev = getattr(_default, "tuning", None)
    set_default_tuning(spec)
    try:
        yield
    finally:
        _default.tuning = prev


def _tuning(tuning):
    """tuning argument -> (use the _tuned entry point?, pointer)."""
    if tuning is None:
        tuning = getattr(_default, "tuning", None)
    elif isinstance(tuning, str):
        tuning = moed_tuning_init(tuning)
    return (tuning is not None), (ctypes.byref(tuning) if tuning is not None else None)


def moed_workspace_bytes(B: int, k: int, H: int, I: int, inter_dtype=torch.float32) -> int:
    """Workspace of moe_decode: the intermediate (256-byte aligned), then B*k*H float32 partials."""
    return int(load().moed_workspace_bytes(B, k, H, I, _DT[inter_dtype]))


_WF = {"mxfp8": 0, "mxfp4": 1}          # moed_wformat


def _kb(K: int, wformat: str) -> int:
    """Code bytes per row of K values."""
    if wformat not in _WF:
        raise ValueError(f"unknown weight format {wformat!r}")
    return K // 2 if wformat == "mxfp4" else K


def moe_decode(x, topk_ids, topk_w, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, out=None,
               out_dtype=torch.bfloat16, inter_dtype=torch.float32, workspace=None, stream=None,
               wformat="mxfp8", tuning=None):
    """The whole layer: returns out [B, H] (out_dtype). wformat: "mxfp8" or "mxfp4"
    (codes [E, I, H/2] and [E, H, I/2], two per byte, low nibble first). tuning: None (the
    built-in table, or the one of an enclosing tuned() block), a spec string or a MoedTuning."""
    B, H = x.shape
    k = topk_ids.shape[1]
    E, I = wg_q.shape[0], wg_q.shape[1]
    HB, IB = _kb(H, wformat), _kb(I, wformat)
    if out is None:
        out = torch.empty((B, H), dtype=out_dtype, device=x.device)
    need = moed_workspace_bytes(B, k, H, I, inter_dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    use, tp = _tuning(tuning)
    lib = load()
    args = (
        _ptr(x, "x", torch.bfloat16, (B, H)), _ptr(topk_ids, "topk_ids", torch.int32, (B, k)),
        _ptr(topk_w, "topk_w", torch.float32, (B, k)),
        _ptr(wg_q, "wg_q", torch.uint8, (E, I, HB)), _ptr(wg_s, "wg_s", torch.uint8, (E, I, H // 32)),
        _ptr(wu_q, "wu_q", torch.uint8, (E, I, HB)), _ptr(wu_s, "wu_s", torch.uint8, (E, I, H // 32)),
        _ptr(wd_q, "wd_q", torch.uint8, (E, H, IB)), _ptr(wd_s, "wd_s", torch.uint8, (E, H, I // 32)),
        _WF[wformat], _ptr(out, "out", None, (B, H)), _DT[out.dtype], _DT[inter_dtype],
        B, E, k, H, I, _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    st = lib.moe_decode_tuned(*args, tp) if use else lib.moe_decode(*args)
    _check(st, "moe_decode")
    return out


def moe_decode_noalloc(x, topk_ids, topk_w, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, out,
                       inter_dtype=torch.float32, stream=None, wformat="mxfp8"):
    """The whole layer into the caller's `out` [B, H] (bf16 or float32) with the library's
    device scratch array instead of a workspace: the call allocates nothing."""
    B, H = x.shape
    k = topk_ids.shape[1]
    E, I = wg_q.shape[0], wg_q.shape[1]
    HB, IB = _kb(H, wformat), _kb(I, wformat)
    st = load().moe_decode_noalloc(
        _ptr(x, "x", torch.bfloat16, (B, H)), _ptr(topk_ids, "topk_ids", torch.int32, (B, k)),
        _ptr(topk_w, "topk_w", torch.float32, (B, k)),
        _ptr(wg_q, "wg_q", torch.uint8, (E, I, HB)), _ptr(wg_s, "wg_s", torch.uint8, (E, I, H // 32)),
        _ptr(wu_q, "wu_q", torch.uint8, (E, I, HB)), _ptr(wu_s, "wu_s", torch.uint8, (E, I, H // 32)),
        _ptr(wd_q, "wd_q", torch.uint8, (E, H, IB)), _ptr(wd_s, "wd_s", torch.uint8, (E, H, I // 32)),
        _WF[wformat], _ptr(out, "out", None, (B, H)), _DT[out.dtype], _DT[inter_dtype],
        B, E, k, H, I, _stream(stream))
    _check(st, "moe_decode_noalloc")
    return out


def moe_decode_gate_up(x, topk_ids, wg_q, wg_s, wu_q, wu_s, a=None, inter_dtype=torch.float32,
                       stream=None, wformat="mxfp8", tuning=None):
    """Gate/up step alone: returns a = SiLU(gate) * up, shape [B, k, I] in the
    library's chunk-interleaved element order (inter_to_bki() gives plain order)."""
    B, H = x.shape
    k = topk_ids.shape[1]
    E, I = wg_q.shape[0], wg_q.shape[1]
    HB = _kb(H, wformat)
    if a is None:
        a = torch.empty((B, k, I), dtype=inter_dtype, device=x.device)
    use, tp = _tuning(tuning)
    lib = load()
    args = (
        _ptr(x, "x", torch.bfloat16, (B, H)), _ptr(topk_ids, "topk_ids", torch.int32, (B, k)),
        _ptr(wg_q, "wg_q", torch.uint8, (E, I, HB)), _ptr(wg_s, "wg_s", torch.uint8, (E, I, H // 32)),
        _ptr(wu_q, "wu_q", torch.uint8, (E, I, HB)), _ptr(wu_s, "wu_s", torch.uint8, (E, I, H // 32)),
        _WF[wformat], _ptr(a, "a", None, (B, k, I)), _DT[a.dtype], B, E, k, H, I, _stream(stream))
    st = lib.moe_decode_gate_up_tuned(*args, tp) if use else lib.moe_decode_gate_up(*args)
    _check(st, "moe_decode_gate_up")
    return a


def moe_decode_down(a, topk_ids, topk_w, wd_q, wd_s, out=None, out_dtype=torch.bfloat16, stream=None,
                    wformat="mxfp8", partials=None, tuning=None):
    """Down step alone: returns out [B, H] from a [B, k, I]. partials: None (one wavefront per
    output) or a float32 CUDA tensor of at least B*k*H elements, which lets batches whose
    tokens share experts take the expert-major form."""
    B, k, I = a.shape
    E, H = wd_q.shape[0], wd_q.shape[1]
    IB = _kb(I, wformat)
    if out is None:
        out = torch.empty((B, H), dtype=out_dtype, device=a.device)
    pp, pn = None, 0
    if partials is not None:
        pp = _ptr(partials, "partials", torch.float32)
        pn = partials.numel() * 4
    use, tp = _tuning(tuning)
    lib = load()
    args = (
        _ptr(a, "a", None, (B, k, I)), _DT[a.dtype], _ptr(topk_ids, "topk_ids", torch.int32, (B, k)),
        _ptr(topk_w, "topk_w", torch.float32, (B, k)),
        _ptr(wd_q, "wd_q", torch.uint8, (E, H, IB)), _ptr(wd_s, "wd_s", torch.uint8, (E, H, I // 32)),
        _WF[wformat], _ptr(out, "out", None, (B, H)), _DT[out.dtype], B, E, k, H, I, pp, pn,
        _stream(stream))
    st = lib.moe_decode_down_tuned(*args, tp) if use else lib.moe_decode_down(*args)
    _check(st, "moe_decode_down")
    return out


def moe_route(logits, k: int, n_shared: int = 0, routed_scale: float = 1.0, ids=None, w=None, stream=None):
    """Router front-end on the GPU: (topk_ids int32 [B, k+n_shared], topk_w float32 [B, k+n_shared])
    from float32 logits [B, E]; shared slots get ids E, E+1, ... and weight 1."""
    B, E = logits.shape
    kt = k + n_shared
    if ids is None:
        ids = torch.empty((B, kt), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((B, kt), dtype=torch.float32, device=logits.device)
    st = load().moe_route(_ptr(logits, "logits", torch.float32, (B, E)), B, E, k, n_shared, float(routed_scale),
                          _ptr(ids, "topk_ids", torch.int32, (B, kt)), _ptr(w, "topk_w", torch.float32, (B, kt)),
                          _stream(stream))
    _check(st, "moe_route")
    return ids, w


# ---------------------------------------------------------------- the block for prompts

def _refuse(t, name, dtypes, shape, dev):
    """Raise what is wrong with an argument of a prompt-side call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a tensor is needed")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported type {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, the call runs on the current device cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous")


# These calls take microseconds on the GPU, so the checks of an argument are one expression, and what is wrong
# is found out only when it fails.
def _arg(t, name, dtypes, shape, dev):
    """Address of a contiguous tensor of one of `dtypes` and of `shape` (None: any) on device index `dev`."""
    try:
        if t.dtype in dtypes and t.get_device() == dev and (shape is None or t.shape == shape) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtypes, shape, dev)


def _opt(t, name, dtypes, shape, dev):
    return None if t is None else _arg(t, name, dtypes, shape, dev)


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, dev):
    if stream is None:
        return _current_raw_stream(dev) if _current_raw_stream else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(shape, dtype, x, stream):
    """A tensor made here for a call on `stream`: its memory is not handed out again before that work is done."""
    # the cheapest of torch's ways: these calls wait for the host as long as for the GPU
    t = torch.empty_like(x) if x.dtype is dtype and x.shape == shape and x.is_contiguous() else x.new_empty(shape, dtype=dtype)
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=x.device)
        here = torch.cuda.current_stream()
        if stream.cuda_stream != here.cuda_stream:
            # the memory may have been an earlier tensor's of the current stream, whose work comes first
            stream.wait_stream(here)
            t.record_stream(stream)
    return t


def _result(t, name, dtypes, shape, dev, dtype, x, stream):
    """(result, address): the caller's tensor, checked, or a new one of `dtype`."""
    if t is None:
        t = _new(shape, dtype, x, stream)
        if t.dtype in dtypes and t.get_device() == dev:
            return t, t.data_ptr()
    return t, _arg(t, name, dtypes, shape, dev)


_U8, _I32, _F32, _BF = (torch.uint8,), (torch.int32,), (torch.float32,), (torch.bfloat16,)
_F = (torch.bfloat16, torch.float32)


def moe_norm(x, gain, residual=None, eps: float = 1e-6, out_dtype=torch.bfloat16, quantize: bool = False, out=None,
             residual_out=None, out_q=None, out_s=None, stream=None):
    """Residual addition and root-mean-square norm: returns (out, residual_out, out_q, out_s).

    out = RMSNorm(x + residual) * gain in out_dtype (None: no plain output); residual_out = x + residual in the
    residual's type (None without a residual; give the residual itself for an update in place); with
    quantize, out_q uint8 [B, H] and out_s uint8 [B, H/32] are the same values in MXFP8, else None."""
    dev = torch.cuda.current_device()
    if x.dim() != 2:
        raise ValueError("x: expected shape [B, H]")
    B, H = x.shape
    if quantize and H % 32:
        raise ValueError("quantize needs H to be a multiple of 32")
    xp, gp, rp, r_dtype = _arg(x, "x", _F, (B, H), dev), _arg(gain, "gain", _F, (H,), dev), None, MOED_BF16
    op = rop = qp = sp = None
    if residual is not None:
        rp, r_dtype = _arg(residual, "residual", _F, (B, H), dev), _DT[residual.dtype]
        residual_out, rop = _result(residual_out, "residual_out", (residual.dtype,), (B, H), dev, residual.dtype, x, stream)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is not None or out_dtype is not None:
        out, op = _result(out, "out", _F, (B, H), dev, out_dtype, x, stream)
    if quantize:
        out_q, qp = _result(out_q, "out_q", _U8, (B, H), dev, torch.uint8, x, stream)
        out_s, sp = _result(out_s, "out_s", _U8, (B, H // 32), dev, torch.uint8, x, stream)
    elif out_q is not None or out_s is not None:
        raise ValueError("out_q and out_s need quantize=True")
    st = load().moe_norm(xp, _DT[x.dtype], rp, r_dtype, gp, _DT[gain.dtype], eps, rop, op,
                         _DT[out.dtype] if out is not None else MOED_BF16, qp, sp, B, H, _raw_stream(stream, dev))
    _check(st, "moe_norm")
    return out, residual_out, out_q, out_s


def moe_group(topk_ids, E: int, order=None, position=None, offsets=None, workspace=None, stream=None):
    """Routed slots sorted by expert: (order int32 [B*k], position int32 [B, k], offsets int32 [E+1])."""
    dev = torch.cuda.current_device()
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids: expected shape [B, k]")
    B, k = topk_ids.shape
    ip = _arg(topk_ids, "topk_ids", _I32, None, dev)
    order, op = _result(order, "order", _I32, (B * k,), dev, torch.int32, topk_ids, stream)
    position, pp = _result(position, "position", _I32, (B, k), dev, torch.int32, topk_ids, stream)
    offsets, fp = _result(offsets, "offsets", _I32, (E + 1,), dev, torch.int32, topk_ids, stream)
    if workspace is None:
        need = int(load().moe_group_workspace_bytes(B, k, E))
        if need:
            workspace = _new((need,), torch.uint8, topk_ids, stream)
    wp = _opt(workspace, "workspace", _U8, None, dev)
    st = load().moe_group(ip, B, k, E, op, pp, fp, wp, 0 if wp is None else workspace.numel(), _raw_stream(stream, dev))
    _check(st, "moe_group")
    return order, position, offsets


def _rows(a, a_s, name, dev, fast):
    """(pointer, scale pointer, moed_rows) of bfloat16 rows, or of MXFP8 codes with their scales."""
    if a.dim() != 2:
        raise ValueError(f"{name}: expected shape [rows, K]")
    if a_s is None:
        if fast:
            raise ValueError(f"fast needs MXFP8 rows ({name}_s)")
        return _arg(a, name, _BF, None, dev), None, MOED_ROWS_BF16
    return (_arg(a, name, _U8, None, dev),
            _arg(a_s, f"{name}_s", _U8, (a.shape[0], a.shape[1] // 32), dev),
            MOED_ROWS_MXFP8_FAST if fast else MOED_ROWS_MXFP8)


def _product_shape(a, offsets, w_q, order):
    if w_q.dim() != 3 or offsets.dim() != 1 or (order is not None and order.dim() != 1):
        raise ValueError("expected weights [E, N, K], offsets [E+1] and order [R]")
    E, N = w_q.shape[0], w_q.shape[1]
    return (order.shape[0] if order is not None else a.shape[0]), E, N, a.shape[1]


def moe_grouped_workspace_bytes(E: int, K: int, N: int, n_a: int, quantized: bool = False, matrices: int = 1) -> int:
    """Workspace of moe_grouped_matmul (matrices 1) or moe_grouped_gate_up (2): 0 where K is a multiple of 128, 512 at least."""
    return int(load().moe_grouped_workspace_bytes(E, K, N, n_a, MOED_ROWS_MXFP8 if quantized else MOED_ROWS_BF16, matrices))


def _product_workspace(workspace, E, K, N, n_a, a_rows, matrices, x, dev, stream):
    need = int(load().moe_grouped_workspace_bytes(E, K, N, n_a, a_rows, matrices))
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _new((need,), torch.uint8, x, stream)
    return _arg(workspace, "workspace", _U8, None, dev), workspace.numel(), workspace


def moe_grouped_gate_up(a, offsets, wg_q, wg_s, wu_q, wu_s, order=None, k: int = 1, a_s=None, out_dtype=torch.bfloat16,
                        quantize: bool = False, out=None, out_s=None, workspace=None, stream=None, wformat="mxfp8",
                        fast: bool = False):
    """SiLU(Wg a) * (Wu a) over the sorted rows of each expert: returns out [R, N] in out_dtype, or with
    quantize (codes uint8 [R, N], scales uint8 [R, N/32]) in MXFP8.

    a: bfloat16 [n, K], or MXFP8 codes uint8 [n, K] with a_s uint8 [n, K/32]. Row r reads a[order[r] // k]
    (order None: a[r]) and belongs to the expert e with offsets[e] <= r < offsets[e+1]; rows from offsets[E] on
    stay as they were. fast (MXFP8 rows, not with float32 outputs): the scaled matrix instructions, which take about
    half the time from 128 rows an expert on and drop 1.5e-5 of the sums, where the others are as good as float32."""
    dev = torch.cuda.current_device()
    ap, asp, a_rows = _rows(a, a_s, "a", dev, fast)
    R, E, N, K = _product_shape(a, offsets, wg_q, order)
    KB = _kb(K, wformat)
    if quantize:
        out = _new((R, N), torch.uint8, a, stream) if out is None else out
        out_s = _new((R, N // 32), torch.uint8, a, stream) if out_s is None else out_s
    elif out_s is not None:
        raise ValueError("out_s needs quantize=True")
    elif out is None:
        out = _new((R, N), out_dtype, a, stream)
    wp, wb, workspace = _product_workspace(workspace, E, K, N, a.shape[0], a_rows, 2, a, dev, stream)
    st = load().moe_grouped_gate_up(
        ap, asp, a_rows, a.shape[0], _opt(order, "order", _I32, (R,), dev), k,
        _arg(offsets, "offsets", _I32, (E + 1,), dev),
        _arg(wg_q, "wg_q", _U8, (E, N, KB), dev), _arg(wg_s, "wg_s", _U8, (E, N, K // 32), dev),
        _arg(wu_q, "wu_q", _U8, (E, N, KB), dev), _arg(wu_s, "wu_s", _U8, (E, N, K // 32), dev),
        _WF[wformat], _arg(out, "out", _U8 if quantize else _F, (R, N), dev),
        _arg(out_s, "out_s", _U8, (R, N // 32), dev) if quantize else None,
        MOED_ROWS_MXFP8 if quantize else _DT[out.dtype], R, E, K, N, wp, wb, _raw_stream(stream, dev))
    _check(st, "moe_grouped_gate_up")
    return (out, out_s) if quantize else out


def moe_grouped_matmul(a, offsets, w_q, w_s, order=None, k: int = 1, a_s=None, out_dtype=torch.bfloat16, out=None,
                       workspace=None, stream=None, wformat="mxfp8", fast: bool = False):
    """W a over the sorted rows of each expert: returns out [R, N] (rows and fast as in moe_grouped_gate_up)."""
    dev = torch.cuda.current_device()
    ap, asp, a_rows = _rows(a, a_s, "a", dev, fast)
    R, E, N, K = _product_shape(a, offsets, w_q, order)
    if out is None:
        out = _new((R, N), out_dtype, a, stream)
    wp, wb, workspace = _product_workspace(workspace, E, K, N, a.shape[0], a_rows, 1, a, dev, stream)
    st = load().moe_grouped_matmul(
        ap, asp, a_rows, a.shape[0], _opt(order, "order", _I32, (R,), dev), k,
        _arg(offsets, "offsets", _I32, (E + 1,), dev),
        _arg(w_q, "w_q", _U8, (E, N, _kb(K, wformat)), dev), _arg(w_s, "w_s", _U8, (E, N, K // 32), dev),
        _WF[wformat], _arg(out, "out", _F, (R, N), dev), _DT[out.dtype], R, E, K, N, wp, wb, _raw_stream(stream, dev))
    _check(st, "moe_grouped_matmul")
    return out


def moe_combine(y, position, topk_w, out=None, out_dtype=torch.bfloat16, stream=None):
    """out[b] = sum_j topk_w[b, j] * y[position[b, j]]: returns out [B, H]."""
    dev = torch.cuda.current_device()
    if y.dim() != 2 or position.dim() != 2:
        raise ValueError("expected y [R, H] and position [B, k]")
    R, H = y.shape
    B, k = position.shape
    yp, pp, wp = (_arg(y, "y", _F, None, dev), _arg(position, "position", _I32, None, dev),
                  _arg(topk_w, "topk_w", _F32, (B, k), dev))
    out, op = _result(out, "out", _F, (B, H), dev, out_dtype, y, stream)
    st = load().moe_combine(yp, _DT[y.dtype], R, pp, wp, op, _DT[out.dtype], B, k, H, _raw_stream(stream, dev))
    _check(st, "moe_combine")
    return out


def moe_prefill_workspace_bytes(B: int, E: int, k: int, H: int, I: int, quantized: bool = False,
                                out_dtype=torch.bfloat16) -> int:
    """Workspace of moe_prefill (quantized: MXFP8 activations)."""
    return int(load().moe_prefill_workspace_bytes(B, E, k, H, I, MOED_ROWS_MXFP8 if quantized else MOED_ROWS_BF16,
                                                  _DT[out_dtype]))


def moe_prefill(x, topk_ids, topk_w, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, x_s=None, out=None,
                out_dtype=torch.bfloat16, workspace=None, stream=None, wformat="mxfp8", fast: bool = False):
    """The whole layer for prompts: returns out [B, H]. x: bfloat16 [B, H], or MXFP8 codes uint8 with x_s
    uint8 [B, H/32] (moe_norm's quantized output). The layer of moe_decode by the grouped products, with two
    more roundings: the intermediate is kept in the type of x (bfloat16 or MXFP8, never float32), and each
    expert's row in out_dtype before the weighted sum (moe_decode sums in float32 and rounds once; so does
    this call with out_dtype float32). fast (with x_s): both products as in moe_grouped_gate_up."""
    dev = torch.cuda.current_device()
    xp, xsp, x_rows = _rows(x, x_s, "x", dev, fast)
    B, H = x.shape
    k = topk_ids.shape[1]
    E, I = wg_q.shape[0], wg_q.shape[1]
    HB, IB = _kb(H, wformat), _kb(I, wformat)
    if out is None:
        out = _new((B, H), out_dtype, x, stream)
    need = moe_prefill_workspace_bytes(B, E, k, H, I, x_s is not None, out.dtype)
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, x, stream)
    st = load().moe_prefill(
        xp, xsp, x_rows, _arg(topk_ids, "topk_ids", _I32, (B, k), dev),
        _arg(topk_w, "topk_w", _F32, (B, k), dev),
        _arg(wg_q, "wg_q", _U8, (E, I, HB), dev), _arg(wg_s, "wg_s", _U8, (E, I, H // 32), dev),
        _arg(wu_q, "wu_q", _U8, (E, I, HB), dev), _arg(wu_s, "wu_s", _U8, (E, I, H // 32), dev),
        _arg(wd_q, "wd_q", _U8, (E, H, IB), dev), _arg(wd_s, "wd_s", _U8, (E, H, I // 32), dev),
        _WF[wformat], _arg(out, "out", _F, (B, H), dev), _DT[out.dtype], B, E, k, H, I,
        _arg(workspace, "workspace", _U8, None, dev), workspace.numel(), _raw_stream(stream, dev))
    _check(st, "moe_prefill")
    return out


def moed_selftest_decode(codes, scales, path: int, out=None, stream=None):
    """Decode codes[t] * 2^(scales[t]-127) with the kernels' decoder; float32 result."""
    n = codes.numel()
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=codes.device)
    st = load().moed_selftest_decode(_ptr(codes, "codes", torch.uint8), _ptr(scales, "scales", torch.uint8),
                                     _ptr(out, "out", torch.float32), n, path, _stream(stream))
    _check(st, "moed_selftest_decode")
    return out


def moed_bench_read(src: torch.Tensor, sink: torch.Tensor, nbytes: int | None = None, stream=None):
    """Stream-read `nbytes` (default: all) of `src` with the contiguous read kernel."""
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(load().moed_bench_read(_ptr(src, "src"), n, _ptr(sink, "sink"), sink.numel() * sink.element_size(),
                                  _stream(stream)), "moed_bench_read")


def moed_bench_read_cfg(src: torch.Tensor, sink: torch.Tensor, nbytes: int, unroll: int, waves_per_group: int,
                        groups: int = 0, stream=None):
    """The read probe with a chosen launch shape (see the header)."""
    _check(load().moed_bench_read_cfg(_ptr(src, "src"), nbytes, _ptr(sink, "sink"), sink.numel() * sink.element_size(),
                                      unroll, waves_per_group, groups, _stream(stream)), "moed_bench_read_cfg")


def moed_bench_copy(src: torch.Tensor, dst: torch.Tensor, nbytes: int | None = None, stream=None):
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    if n > dst.numel() * dst.element_size():
        raise ValueError("moed_bench_copy: dst too small")
    _check(load().moed_bench_copy(_ptr(src, "src"), _ptr(dst, "dst"), n, _stream(stream)), "moed_bench_copy")


def moed_status_string(status: int) -> str:
    return load().moed_status_string(status).decode()


def moed_last_hip_error() -> int:
    return load().moed_last_hip_error()


def inter_to_bki(a: torch.Tensor) -> torch.Tensor:
    """Reorder the library's chunk-interleaved intermediate (see the header) to plain [B, k, I]."""
    B, k, I = a.shape
    q, per = (2, 8) if a.dtype == torch.bfloat16 else (4, 4)
    return a.reshape(B * k, q, I // 16, per).permute(0, 2, 1, 3).reshape(B, k, I)


def layer_device_inputs(L, device="cuda"):
    """Host parts of a synth.LayerInputs -> device tensors (x bf16, ids int32, w f32)."""
    x = torch.from_numpy(L.x.view("int16")).view(torch.bfloat16).to(device)
    ids = torch.from_numpy(L.ids).to(device)
    w = torch.from_numpy(L.w).to(device)
    return x, ids, w
