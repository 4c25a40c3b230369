"""ctypes binding of libbfq (include/bfq.h): the same entry-point names, argument marshalling
only. Every step of the computation runs in the HIP kernels of libbfq.so; PyTorch supplies
device memory (tensor.data_ptr()) and the current HIP stream. There is no fallback: if the
library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
# BFQ_LIBRARY names another build of the same library (for example one whose host code is
# built with sanitizers); by default the in-tree libbfq.so.
LIB_PATH = os.environ.get("BFQ_LIBRARY") or os.path.join(HERE, "libbfq.so")

# status codes (bfq_status)
BFQ_OK = 0
BFQ_WARN_DEFAULT_TILE = 1
BFQ_ERR_NULL = -1
BFQ_ERR_SHAPE = -2
BFQ_ERR_DTYPE = -3
BFQ_ERR_ALIGN = -4
BFQ_ERR_WORKSPACE = -5
BFQ_ERR_TILE = -6
BFQ_ERR_TABLE = -7
BFQ_ERR_HIP = -8
BFQ_ERR_ARG = -9

# dtypes (bfq_dtype)
BFQ_BF16, BFQ_FP16, BFQ_FP32, BFQ_E4M3FN, BFQ_INT8, BFQ_INT32 = range(6)
# scale layouts (bfq_scale_layout)
BFQ_SCALES_ROW_MAJOR = 0
BFQ_SCALES_COL_MAJOR = 1
BFQ_SCALES_PACKED_UE8M0 = 2   # uint32 words of four E8M0 codes (UE8M0 scales only)
# weight-code layouts (bfq_weight_layout)
BFQ_W_ROW_MAJOR = 0
BFQ_W_PACKED16 = 1
# scale formats (bfq_scale_format)
BFQ_SCALE_FP32 = 0
BFQ_SCALE_UE8M0 = 1

# activations of the gated product (bfq_activation)
BFQ_ACT_SILU = 0
BFQ_ACT_GELU_TANH = 1
# what one gate value of the norm step covers (bfq_gate_kind)
BFQ_GATE_NONE, BFQ_GATE_CHANNEL, BFQ_GATE_TOKEN, BFQ_GATE_FULL = range(4)

DEFAULT_EPS = 1e-10
NORM_EPS = 1e-6
# Maximum K of the norm step (a row stays in a workgroup's registers).
NORM_MAX_K = 16384
BLOCK_SHAPE = (128, 128)
# Maximum K of the per-token x per-channel format (block_shape (1, K)).
CHANNEL_MAX_K = 32768


def channel_block_shape(K: int):
    """block_shape of the per-token x per-channel format (one scale per token and per output
    channel; Helion linear-backend page, scope section)."""
    return (1, int(K))

EXPORTED = (
    "bfq_quant_tokens", "bfq_quant_weight_blocks", "bfq_pack_weights", "bfq_select_tile",
    "bfq_gemm_workspace_bytes", "bfq_block_gemm", "bfq_load_tile_table",
    "bfq_num_tile_candidates", "bfq_get_tile_candidate", "bfq_status_string",
    "bfq_last_error", "bfq_debug_block_partials_i32", "bfq_debug_encode",
    "bfq_set_batch_invariant", "bfq_get_batch_invariant",
    "bfq_moe_align_workspace_bytes", "bfq_moe_align", "bfq_moe_select_tile",
    "bfq_moe_gemm_workspace_bytes", "bfq_moe_block_gemm", "bfq_moe_num_tile_candidates",
    "bfq_moe_get_tile_candidate", "bfq_block_gemm_noalloc", "bfq_noalloc_scratch_bytes",
    "bfq_probe_mfma_peak", "bfq_probe_mfma_flops",
    "bfq_gated_gemm", "bfq_gated_select_tile", "bfq_gated_gemm_workspace_bytes",
    "bfq_gated_num_tile_candidates", "bfq_gated_get_tile_candidate", "bfq_gated_backward",
    "bfq_transpose_weights", "bfq_norm_residual", "bfq_norm_residual_backward",
    "bfq_norm_residual_backward_workspace_bytes",
)


class bfq_tile(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("bm", ctypes.c_int32), ("bn", ctypes.c_int32),
                ("bk", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("waves_m", ctypes.c_int32), ("waves_n", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("group_m", ctypes.c_int32),
                ("sched", ctypes.c_int32), ("raster", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]

    FIELDS = ("variant", "bm", "bn", "bk", "split_k", "waves_m", "waves_n", "stages", "group_m",
              "sched", "raster")

    def as_dict(self) -> dict:
        return {f: int(getattr(self, f)) for f in self.FIELDS}

    @classmethod
    def from_dict(cls, d: dict) -> "bfq_tile":
        t = cls()
        t.bk = 128
        t.split_k = 1
        t.waves_m = 1
        t.stages = 2
        t.group_m = 1
        for k, v in d.items():
            if k in cls.FIELDS:
                setattr(t, k, int(v))
        return t


class BfqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}: {last_error()}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libbfq.so not found at {LIB_PATH}; build it with "
            "`python -m block_scaled_w8a8_amd.build` (hipcc, gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                            ctypes.c_size_t)
    tp = ctypes.POINTER(bfq_tile)
    bs = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "bfq_quant_tokens": (i32, [p, i64, i64, i32, i32, p, p, i32, i64, f32, i32, p]),
        "bfq_quant_weight_blocks": (i32, [p, i64, i64, bs, i32, p, p, f32, i32, p]),
        "bfq_pack_weights": (i32, [p, i64, i64, i32, p, p]),
        "bfq_select_tile": (i32, [i64, i64, i64, bs, i32, i32, i32, i32, tp]),
        "bfq_gemm_workspace_bytes": (sz, [i64, i64, i64, tp]),
        "bfq_block_gemm": (i32, [p, p, i32, i64, p, p, i32, i32, p, i64, i64, i64, bs, i32, i32,
                                 tp, p, sz, p]),
        "bfq_load_tile_table": (i32, [ctypes.c_char_p]),
        "bfq_num_tile_candidates": (i32, [bs, i32, i32, i32]),
        "bfq_get_tile_candidate": (i32, [bs, i32, i32, i32, i32, tp]),
        "bfq_status_string": (ctypes.c_char_p, [i32]),
        "bfq_last_error": (ctypes.c_char_p, []),
        "bfq_debug_block_partials_i32": (i32, [p, p, p, i64, i64, i64, p]),
        "bfq_debug_encode": (i32, [p, i64, i32, p, p]),
        "bfq_set_batch_invariant": (None, [i32]),
        "bfq_moe_align_workspace_bytes": (sz, [i64, i32, i32]),
        "bfq_moe_align": (i32, [p, i64, i32, i32, p, p, p, sz, p]),
        "bfq_moe_select_tile": (i32, [i64, i32, i32, i64, i64, bs, i32, i32, i32, i32, tp]),
        "bfq_moe_gemm_workspace_bytes": (sz, [i64, i32, i64, tp]),
        "bfq_moe_block_gemm": (i32, [p, p, i32, i64, p, p, i32, p, p, i32, i32, p, i64, i64, i64,
                                     i32, bs, i32, i32, tp, p, sz, p]),
        "bfq_moe_num_tile_candidates": (i32, [i32, i32]),
        "bfq_moe_get_tile_candidate": (i32, [i32, i32, i32, tp]),
        "bfq_get_batch_invariant": (i32, []),
        "bfq_block_gemm_noalloc": (i32, [p, p, i32, i64, p, p, i32, i32, p, i64, i64, i64, bs,
                                         i32, i32, tp, p]),
        "bfq_noalloc_scratch_bytes": (sz, []),
        "bfq_probe_mfma_peak": (i32, [i64, i64, p, p]),
        "bfq_probe_mfma_flops": (ctypes.c_double, [i64, i64]),
        "bfq_gated_gemm": (i32, [p, p, i32, i64, p, p, i32, i32, i32, p, p, i32, i64, f32, p, i64,
                                 i64, i64, bs, i32, i32, tp, p, sz, p]),
        "bfq_gated_select_tile": (i32, [i64, i64, i64, i32, i32, i32, tp]),
        "bfq_gated_gemm_workspace_bytes": (sz, [i64, i64, i64, i32, i32, i32, tp]),
        "bfq_gated_num_tile_candidates": (i32, [i32, i32]),
        "bfq_gated_get_tile_candidate": (i32, [i32, i32, i32, tp]),
        "bfq_gated_backward": (i32, [p, p, i32, p, p, i32, p, i32, i64, f32, i32, p, i64, i64, p]),
        "bfq_transpose_weights": (i32, [p, p, i64, i64, i32, p, p, p]),
        "bfq_norm_residual": (i32, [p, p, i32, p, p, i32, f32, p, f32, p, p, p, i32, i32, p, i32,
                                    i64, f32, i32, i64, i64, p]),
        "bfq_norm_residual_backward_workspace_bytes": (sz, [i64, i64]),
        "bfq_norm_residual_backward": (i32, [p, p, i32, p, p, i32, f32, p, f32, p, p, p, p, p, p, p,
                                             i64, i64, p, sz, p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()

_warned: set = set()


def status_string(s: int) -> str:
    return lib.bfq_status_string(int(s)).decode()


def last_error() -> str:
    return lib.bfq_last_error().decode()


def _check(status: int, where: str, warn_key=None, depth=3) -> int:
    if status < 0:
        raise BfqError(status, where)
    if status > 0 and warn_key not in _warned:
        _warned.add(warn_key)
        warnings.warn(f"{where}: {status_string(status)} (no tuned tile for {warn_key}; "
                      "using the default tile)", RuntimeWarning, stacklevel=depth)   # the caller's line
    return status


_BLOCK_128 = (ctypes.c_int32 * 2)(*BLOCK_SHAPE)      # read only by the library


def _block_shape(block_shape=BLOCK_SHAPE):
    return _BLOCK_128 if block_shape is BLOCK_SHAPE else (ctypes.c_int32 * 2)(*block_shape)


def _ptr(t) -> int:
    """Device address of a tensor (or an int address / None)."""
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


# ------------------------------------------------------------------ argument checks
# The kernels take raw device addresses and assume the layouts stated in include/bfq.h (rows
# of codes and outputs packed at stride K or N, scales at the stated leading dimension). The
# wrappers below check every tensor against those assumptions before the C call, so that a
# host tensor, a strided view or a buffer of the wrong size raises here instead of handing a
# kernel an address it would read or write past. Order: type, dtype, shape, strides, device
# (a tensor that passes all but the device check is a host tensor). Plain int addresses are
# passed through unchecked: the caller vouches for them.

class BfqArgumentError(ValueError):
    """A tensor argument does not match what the kernel will read or write."""


U8_CODES = ("uint8", "float8_e4m3fn")


_torch = None          # torch, once a tensor has been seen (importing the binding does not need it)
_Tensor = None         # torch.Tensor, likewise
_DTYPE_NAMES: dict = {}
_DTYPE_SETS: dict = {}  # tuples of dtype names -> the torch dtypes they name


def _torch_module():
    global _torch, _Tensor
    if _torch is None:
        import torch
        _torch, _Tensor = torch, torch.Tensor
    return _torch


def _dt(t) -> str:
    name = _DTYPE_NAMES.get(t.dtype)
    if name is None:
        name = _DTYPE_NAMES[t.dtype] = str(t.dtype).replace("torch.", "")
    return name


def _is(t, dtypes) -> bool:
    """A plain tensor of one of these types (what a call is usually given); anything else goes
    through the checks that say what is wrong."""
    if t.__class__ is not _Tensor:
        return False
    known = _DTYPE_SETS.get(dtypes)
    if known is None:
        known = _DTYPE_SETS[dtypes] = frozenset(getattr(_torch, n) for n in dtypes)
    return t.dtype in known


def _tensor(t, name, dtypes):
    if isinstance(t, int):
        return False
    if not isinstance(t, (_torch or _torch_module()).Tensor):
        raise BfqArgumentError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if _dt(t) not in dtypes:
        raise BfqArgumentError(f"{name} has dtype {_dt(t)}; expected one of {', '.join(dtypes)}")
    return True


def _devices(**tensors):
    """Last check of a wrapper: every tensor argument is on the current GPU."""
    cur = None
    for name, t in tensors.items():
        if t is not None and not isinstance(t, int):
            dev = t.get_device()
            if dev < 0:
                raise BfqArgumentError(f"{name} is on device {t.device}; the kernels need a GPU tensor")
            if cur is None:                    # a GPU tensor exists, so the runtime is initialised
                cur = (_torch or _torch_module())._C._cuda_getDevice()
            if dev != cur:
                raise BfqArgumentError(f"{name} is on {t.device}, not the current device cuda:{cur}")


def _rows(t, name, dtypes, rows, cols):
    """A [rows, cols] matrix whose rows are packed at stride cols (what the kernels index)."""
    if _is(t, dtypes) and t.is_contiguous() and t.shape == (rows, cols):
        return
    if not _tensor(t, name, dtypes):
        return
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise BfqArgumentError(f"{name} has shape {tuple(shape)}; expected ({rows}, {cols})")
    if not t.is_contiguous() and rows > 0 and cols > 0 and (
            t.stride(1) != 1 or (rows > 1 and t.stride(0) != cols)):
        raise BfqArgumentError(f"{name} has strides {t.stride()}; its rows must be contiguous "
                               f"at stride {cols} (call .contiguous())")


def _flat(t, name, dtypes, numel, exact=True):
    """A contiguous buffer of exactly (or at least) numel elements, any shape."""
    if _is(t, dtypes) and t.numel() == numel and t.is_contiguous():
        return
    if not _tensor(t, name, dtypes):
        return
    if (t.numel() != numel) if exact else (t.numel() < numel):
        raise BfqArgumentError(f"{name} holds {t.numel()} elements; expected "
                               f"{'' if exact else 'at least '}{numel}")
    if not t.is_contiguous():
        raise BfqArgumentError(f"{name} must be contiguous")


def _scales(t, name, layout, ld, m, groups, write):
    """Activation scales in `layout` with leading dimension ld over m tokens and `groups`
    scales per token: the 2-D view must cover every element the kernel touches, at stride
    (ld, 1). Packed words: int32, ceil(groups/4) word rows of ld words, ld >= m rounded up to
    4 when the quantizer writes them (>= m when the GEMM reads them)."""
    if layout == BFQ_SCALES_PACKED_UE8M0:
        if not _tensor(t, name, ("int32", "uint32")):
            return
        need = ((groups + 3) // 4, (m + 3) // 4 * 4 if write else m)
    else:
        if not _tensor(t, name, ("float32",)):
            return
        need = (m, groups) if layout == BFQ_SCALES_ROW_MAJOR else (groups, m)
    shape = t.shape
    if len(shape) != 2:
        raise BfqArgumentError(f"{name} must be 2-D, got shape {tuple(shape)}")
    if shape[0] < need[0] or shape[1] < need[1]:
        raise BfqArgumentError(f"{name} has shape {tuple(shape)}; the layout needs at least "
                               f"{need}")
    if shape[0] > 1 and t.stride(0) != ld:
        raise BfqArgumentError(f"{name} has row stride {t.stride(0)} but scale_ld is {ld}")
    if shape[1] > 1 and t.stride(1) != 1:
        raise BfqArgumentError(f"{name} must have unit stride along its second dimension")


def _workspace(t, nbytes):
    if t is None or isinstance(t, int):
        return
    if not isinstance(t, (_torch or _torch_module()).Tensor):
        raise BfqArgumentError("workspace must be a torch.Tensor")
    if t.numel() * t.element_size() < nbytes or not t.is_contiguous():
        raise BfqArgumentError(f"workspace holds {t.numel() * t.element_size()} bytes "
                               f"(contiguous: {t.is_contiguous()}); {nbytes} are declared")


CODE_DTYPES = U8_CODES + ("int8",)
OUT_DTYPES = ("bfloat16", "float16", "float32")


def _shape2(t, name):
    if t.__class__ is _Tensor:
        shape = t.shape
        if len(shape) == 2:
            return shape
    shape = getattr(t, "shape", ())
    if not hasattr(t, "dim") or len(shape) != 2:
        raise BfqArgumentError(f"{name} must be a 2-D tensor")
    return int(shape[0]), int(shape[1])


def _same_codes(a, w):
    """Token and weight codes must be the same code type (e4m3fn bytes or int8)."""
    if isinstance(a, int) or isinstance(w, int):
        return
    if (_dt(a) == "int8") != (_dt(w) == "int8"):
        raise BfqArgumentError(f"a_q ({_dt(a)}) and w_q ({_dt(w)}) hold different code types")


def _stream(stream):
    if stream is None:
        torch = _torch or _torch_module()
        if not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        # the handle, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream if isinstance(stream, int) else stream.cuda_stream


_CODE_TYPES = {"uint8": BFQ_E4M3FN, "float8_e4m3fn": BFQ_E4M3FN, "int8": BFQ_INT8}
_OUT_TYPES = {"bfloat16": BFQ_BF16, "float16": BFQ_FP16, "float32": BFQ_FP32}


def _qdtype(t) -> int:
    q = _CODE_TYPES.get(_dt(t))
    if q is None:
        raise BfqArgumentError(f"code tensor dtype {t.dtype} is neither e4m3fn/uint8 nor int8")
    return q


def _odtype(t) -> int:
    return _OUT_TYPES[_dt(t)]


# ----------------------------------------------------------------------- entry points

def bfq_quant_tokens(x, q, scales, layout=BFQ_SCALES_ROW_MAJOR, scale_ld=None,
                     eps=DEFAULT_EPS, group_size=128, stream=None,
                     scale_fmt=BFQ_SCALE_FP32) -> int:
    """x: bf16 [M, K]; q: uint8/float8_e4m3fn (e4m3fn codes) or int8 [M, K];
    scales: fp32, [M, ld] (row-major) or [K/group_size, ld] (column-major). group_size 128,
    or K for one scale per token."""
    M, K = _shape2(x, "x")
    if scale_ld is None:
        scale_ld = scales.stride(0)
    _rows(x, "x", ("bfloat16",), M, K)
    _rows(q, "q", CODE_DTYPES, M, K)
    if group_size > 0 and K % group_size == 0:
        _scales(scales, "scales", layout, scale_ld, M, K // group_size, write=True)
    _devices(x=x, q=q, scales=scales)
    st = lib.bfq_quant_tokens(_ptr(x), M, K, group_size, _qdtype(q), _ptr(q), _ptr(scales),
                              layout, scale_ld, eps, scale_fmt, _stream(stream))
    return _check(st, "bfq_quant_tokens")


def bfq_quant_weight_blocks(w, q, scales, eps=DEFAULT_EPS, block_shape=BLOCK_SHAPE,
                            stream=None, scale_fmt=BFQ_SCALE_FP32) -> int:
    """w: fp32 [N, K]; q: codes [N, K]; scales: fp32 [N/128, K/128], or [N] (any shape of N
    contiguous floats) with block_shape (1, K)."""
    N, K = _shape2(w, "w")
    _rows(w, "w", ("float32",), N, K)
    _rows(q, "q", CODE_DTYPES, N, K)
    per_channel = tuple(block_shape)[0] == 1
    _flat(scales, "scales", ("float32",), N if per_channel else (N // 128) * (K // 128))
    _devices(w=w, q=q, scales=scales)
    st = lib.bfq_quant_weight_blocks(_ptr(w), N, K, _block_shape(block_shape), _qdtype(q),
                                     _ptr(q), _ptr(scales), eps, scale_fmt, _stream(stream))
    return _check(st, "bfq_quant_weight_blocks")


def bfq_pack_weights(w_q, w_packed, stream=None) -> int:
    """w_q: row-major codes [N, K]; w_packed: a separate N*K-byte buffer (any shape with that
    many bytes, e.g. [N, K] uint8) that receives the BFQ_W_PACKED16 layout."""
    N, K = _shape2(w_q, "w_q")
    _rows(w_q, "w_q", CODE_DTYPES, N, K)
    if _tensor(w_packed, "w_packed", CODE_DTYPES):
        if w_packed.numel() * w_packed.element_size() != N * K or not w_packed.is_contiguous():
            raise BfqArgumentError("w_packed must be a contiguous buffer of exactly N*K bytes")
    _devices(w_q=w_q, w_packed=w_packed)
    st = lib.bfq_pack_weights(_ptr(w_q), N, K, _qdtype(w_q), _ptr(w_packed), _stream(stream))
    return _check(st, "bfq_pack_weights")


def bfq_select_tile(M, N, K, in_dtype=BFQ_E4M3FN, out_dtype=BFQ_BF16,
                    block_shape=BLOCK_SHAPE, w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32):
    """Returns (status, bfq_tile)."""
    t = bfq_tile()
    st = lib.bfq_select_tile(M, N, K, _block_shape(block_shape), in_dtype, out_dtype,
                             w_layout, scale_fmt, ctypes.byref(t))
    if st < 0:
        raise BfqError(st, "bfq_select_tile")
    return st, t


def bfq_gemm_workspace_bytes(M, N, K, tile=None) -> int:
    return int(lib.bfq_gemm_workspace_bytes(M, N, K, ctypes.byref(tile) if tile else None))


def bfq_block_gemm(a_q, a_scales, w_q, w_scales, out, a_layout=BFQ_SCALES_ROW_MAJOR,
                   a_scale_ld=None, tile=None, workspace=None, workspace_bytes=None,
                   block_shape=BLOCK_SHAPE, stream=None, w_layout=BFQ_W_ROW_MAJOR,
                   scale_fmt=BFQ_SCALE_FP32) -> int:
    """a_q [M, K] codes, w_q [N, K] codes in w_layout (row-major, or packed by
    bfq_pack_weights and still shaped [N, K]), a_scales per layout, w_scales [N/128, K/128],
    out [M, N] (bf16 / fp16 / fp32). scale_fmt BFQ_SCALE_UE8M0 declares every scale a power
    of two. block_shape (1, K): per-token a_scales ([M, 1] or [1, M]) and per-channel
    w_scales [N]. Returns the status (>= 0)."""
    M, K = _shape2(a_q, "a_q")
    N = _shape2(w_q, "w_q")[0]
    if a_scale_ld is None:
        a_scale_ld = a_scales.stride(0)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _rows(a_q, "a_q", CODE_DTYPES, M, K)
    _rows(w_q, "w_q", CODE_DTYPES, N, K)
    _same_codes(a_q, w_q)
    per_channel = tuple(block_shape)[0] == 1
    _scales(a_scales, "a_scales", a_layout, a_scale_ld, M, 1 if per_channel else K // 128,
            write=False)
    _flat(w_scales, "w_scales", ("float32",), N if per_channel else (N // 128) * (K // 128))
    _rows(out, "out", OUT_DTYPES, M, N)
    _workspace(workspace, workspace_bytes)
    _devices(a_q=a_q, a_scales=a_scales, w_q=w_q, w_scales=w_scales, out=out, workspace=workspace)
    st = lib.bfq_block_gemm(_ptr(a_q), _ptr(a_scales), a_layout, a_scale_ld, _ptr(w_q),
                            _ptr(w_scales), w_layout, scale_fmt, _ptr(out), M, N, K,
                            _block_shape(block_shape),
                            _qdtype(a_q), _odtype(out), ctypes.byref(tile) if tile else None,
                            _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "bfq_block_gemm", warn_key=(N, K))


def bfq_block_gemm_noalloc(a_q, a_scales, w_q, w_scales, out, a_layout=BFQ_SCALES_ROW_MAJOR,
                           a_scale_ld=None, tile=None, block_shape=BLOCK_SHAPE, stream=None,
                           w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32) -> int:
    """bfq_block_gemm without a workspace argument: split-K partials and stream-K slots use the
    library's static device buffer (bfq_noalloc_scratch_bytes()). No allocation anywhere on
    this path; calls that overlap on one GPU race."""
    M, K = _shape2(a_q, "a_q")
    N = _shape2(w_q, "w_q")[0]
    if a_scale_ld is None:
        a_scale_ld = a_scales.stride(0)
    _rows(a_q, "a_q", CODE_DTYPES, M, K)
    _rows(w_q, "w_q", CODE_DTYPES, N, K)
    _same_codes(a_q, w_q)
    per_channel = tuple(block_shape)[0] == 1
    _scales(a_scales, "a_scales", a_layout, a_scale_ld, M, 1 if per_channel else K // 128,
            write=False)
    _flat(w_scales, "w_scales", ("float32",), N if per_channel else (N // 128) * (K // 128))
    _rows(out, "out", OUT_DTYPES, M, N)
    _devices(a_q=a_q, a_scales=a_scales, w_q=w_q, w_scales=w_scales, out=out)
    st = lib.bfq_block_gemm_noalloc(_ptr(a_q), _ptr(a_scales), a_layout, a_scale_ld, _ptr(w_q),
                                    _ptr(w_scales), w_layout, scale_fmt, _ptr(out), M, N, K,
                                    _block_shape(block_shape), _qdtype(a_q), _odtype(out),
                                    ctypes.byref(tile) if tile else None, _stream(stream))
    return _check(st, "bfq_block_gemm_noalloc", warn_key=(N, K))


def bfq_noalloc_scratch_bytes() -> int:
    return int(lib.bfq_noalloc_scratch_bytes())


def bfq_load_tile_table(path=None) -> int:
    st = lib.bfq_load_tile_table(path.encode() if path else None)
    return _check(st, "bfq_load_tile_table")


def bfq_num_tile_candidates(in_dtype=BFQ_E4M3FN, w_layout=BFQ_W_ROW_MAJOR,
                            scale_fmt=BFQ_SCALE_FP32, block_shape=BLOCK_SHAPE) -> int:
    return int(lib.bfq_num_tile_candidates(_block_shape(block_shape), in_dtype, w_layout,
                                           scale_fmt))


def bfq_get_tile_candidate(index, in_dtype=BFQ_E4M3FN, w_layout=BFQ_W_ROW_MAJOR,
                           scale_fmt=BFQ_SCALE_FP32, block_shape=BLOCK_SHAPE) -> bfq_tile:
    t = bfq_tile()
    _check(lib.bfq_get_tile_candidate(_block_shape(block_shape), in_dtype, w_layout, scale_fmt,
                                      index, ctypes.byref(t)),
           "bfq_get_tile_candidate")
    return t


def bfq_moe_align(topk_ids, E, expert_offsets, sorted_pairs, workspace=None, stream=None) -> int:
    """topk_ids int32 [T, topk]; expert_offsets int32 [E+1]; sorted_pairs int32 [T*topk]."""
    T, topk = _shape2(topk_ids, "topk_ids")
    need = int(lib.bfq_moe_align_workspace_bytes(T, topk, E))
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _rows(topk_ids, "topk_ids", ("int32",), T, topk)
    _flat(expert_offsets, "expert_offsets", ("int32",), E + 1)
    _flat(sorted_pairs, "sorted_pairs", ("int32",), T * topk, exact=False)
    _workspace(workspace, need)
    _devices(topk_ids=topk_ids, expert_offsets=expert_offsets, sorted_pairs=sorted_pairs,
             workspace=workspace)
    st = lib.bfq_moe_align(_ptr(topk_ids), T, topk, E, _ptr(expert_offsets), _ptr(sorted_pairs),
                           _ptr(workspace), wb if workspace is not None else need, _stream(stream))
    return _check(st, "bfq_moe_align")


def bfq_moe_select_tile(T, topk, E, N, K, out_dtype=BFQ_BF16, w_layout=BFQ_W_ROW_MAJOR,
                        scale_fmt=BFQ_SCALE_FP32):
    """Returns (status, bfq_tile)."""
    t = bfq_tile()
    st = lib.bfq_moe_select_tile(T, topk, E, N, K, _block_shape(BLOCK_SHAPE), BFQ_E4M3FN,
                                 out_dtype, w_layout, scale_fmt, ctypes.byref(t))
    if st < 0:
        raise BfqError(st, "bfq_moe_select_tile")
    return st, t


def bfq_moe_gemm_workspace_bytes(T, topk, N, tile) -> int:
    return int(lib.bfq_moe_gemm_workspace_bytes(T, topk, N, ctypes.byref(tile)))


def bfq_moe_block_gemm(a_q, a_scales, sorted_pairs, expert_offsets, topk, w_q, w_scales, out,
                       a_layout=BFQ_SCALES_ROW_MAJOR, a_scale_ld=None, tile=None, workspace=None,
                       workspace_bytes=None, stream=None, w_layout=BFQ_W_ROW_MAJOR,
                       scale_fmt=BFQ_SCALE_FP32) -> int:
    """a_q [T, K]; w_q [E, N, K] (row-major, or each expert packed); w_scales
    [E, N/128, K/128]; out [T*topk, N] in pair order."""
    T, K = _shape2(a_q, "a_q")
    if not hasattr(w_q, "dim") or w_q.dim() != 3:
        raise BfqArgumentError("w_q must be a 3-D [E, N, K] tensor")
    E, N = w_q.shape[0], w_q.shape[1]
    if a_scale_ld is None:
        a_scale_ld = a_scales.stride(0)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _rows(a_q, "a_q", U8_CODES, T, K)
    if w_q.shape[2] != K:
        raise BfqArgumentError(f"w_q has shape {tuple(w_q.shape)}; its last dimension must be K={K}")
    _flat(w_q, "w_q", U8_CODES, E * N * K)
    _scales(a_scales, "a_scales", a_layout, a_scale_ld, T, K // 128, write=False)
    _flat(w_scales, "w_scales", ("float32",), E * (N // 128) * (K // 128))
    _flat(sorted_pairs, "sorted_pairs", ("int32",), T * topk, exact=False)
    _flat(expert_offsets, "expert_offsets", ("int32",), E + 1)
    _rows(out, "out", OUT_DTYPES, T * topk, N)
    _workspace(workspace, workspace_bytes)
    _devices(a_q=a_q, a_scales=a_scales, sorted_pairs=sorted_pairs,
             expert_offsets=expert_offsets, w_q=w_q, w_scales=w_scales, out=out,
             workspace=workspace)
    st = lib.bfq_moe_block_gemm(_ptr(a_q), _ptr(a_scales), a_layout, a_scale_ld, _ptr(sorted_pairs),
                                _ptr(expert_offsets), topk, _ptr(w_q), _ptr(w_scales), w_layout,
                                scale_fmt, _ptr(out), T, N, K, E, _block_shape(BLOCK_SHAPE),
                                BFQ_E4M3FN, _odtype(out), ctypes.byref(tile) if tile else None,
                                _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "bfq_moe_block_gemm", warn_key=("moe", E, N, K))


def bfq_moe_num_tile_candidates(w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32) -> int:
    return int(lib.bfq_moe_num_tile_candidates(w_layout, scale_fmt))


def bfq_moe_get_tile_candidate(index, w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32) -> bfq_tile:
    t = bfq_tile()
    _check(lib.bfq_moe_get_tile_candidate(w_layout, scale_fmt, index, ctypes.byref(t)),
           "bfq_moe_get_tile_candidate")
    return t


def bfq_status_string(s: int) -> str:
    return status_string(s)


def bfq_set_batch_invariant(enable: bool) -> None:
    lib.bfq_set_batch_invariant(1 if enable else 0)


def bfq_get_batch_invariant() -> bool:
    return bool(lib.bfq_get_batch_invariant())


def bfq_last_error() -> str:
    return last_error()


def bfq_debug_block_partials_i32(a_q, w_q, partials, stream=None) -> int:
    M, K = _shape2(a_q, "a_q")
    N = _shape2(w_q, "w_q")[0]
    _rows(a_q, "a_q", ("int8",), M, K)
    _rows(w_q, "w_q", ("int8",), N, K)
    _flat(partials, "partials", ("int32",), (K // 128) * M * N)
    _devices(a_q=a_q, w_q=w_q, partials=partials)
    st = lib.bfq_debug_block_partials_i32(_ptr(a_q), _ptr(w_q), _ptr(partials), M, N, K,
                                          _stream(stream))
    return _check(st, "bfq_debug_block_partials_i32")


def bfq_probe_mfma_peak(blocks, iters, out, stream=None) -> float:
    """Launch the MFMA-only probe (out: >= blocks * 512 fp32 on the device); returns the
    flops of the launch."""
    _flat(out, "out", ("float32",), blocks * 512, exact=False)
    _devices(out=out)
    _check(lib.bfq_probe_mfma_peak(blocks, iters, _ptr(out), _stream(stream)),
           "bfq_probe_mfma_peak")
    return float(lib.bfq_probe_mfma_flops(blocks, iters))


def bfq_debug_encode(x, codes, q_dtype=BFQ_E4M3FN, stream=None) -> int:
    _flat(x, "x", ("float32",), x.numel())
    _flat(codes, "codes", CODE_DTYPES, x.numel())
    _devices(x=x, codes=codes)
    st = lib.bfq_debug_encode(_ptr(x), x.numel(), q_dtype, _ptr(codes), _stream(stream))
    return _check(st, "bfq_debug_encode")


# ------------------------------------------------------------- feed-forward operators

def _workspace_arg(workspace, workspace_bytes):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return workspace_bytes


def bfq_gated_select_tile(M, F, K, out_dtype=BFQ_BF16, w_layout=BFQ_W_ROW_MAJOR,
                          scale_fmt=BFQ_SCALE_FP32) -> bfq_tile:
    """The tile bfq_gated_gemm takes (bn = output columns of a workgroup)."""
    t = bfq_tile()
    _check(lib.bfq_gated_select_tile(M, F, K, out_dtype, w_layout, scale_fmt, ctypes.byref(t)),
           "bfq_gated_select_tile")
    return t


def bfq_gated_gemm_workspace_bytes(M, F, K, out_dtype=BFQ_BF16, w_layout=BFQ_W_ROW_MAJOR,
                                   scale_fmt=BFQ_SCALE_FP32, tile=None) -> int:
    return int(lib.bfq_gated_gemm_workspace_bytes(M, F, K, out_dtype, w_layout, scale_fmt,
                                                  ctypes.byref(tile) if tile else None))


def bfq_gated_num_tile_candidates(w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32) -> int:
    return int(lib.bfq_gated_num_tile_candidates(w_layout, scale_fmt))


def bfq_gated_get_tile_candidate(index, w_layout=BFQ_W_ROW_MAJOR,
                                 scale_fmt=BFQ_SCALE_FP32) -> bfq_tile:
    t = bfq_tile()
    _check(lib.bfq_gated_get_tile_candidate(w_layout, scale_fmt, index, ctypes.byref(t)),
           "bfq_gated_get_tile_candidate")
    return t


def bfq_gated_gemm(a_q, a_scales, w_q, w_scales, out, act=BFQ_ACT_SILU,
                   a_layout=BFQ_SCALES_ROW_MAJOR, a_scale_ld=None, out_scales=None,
                   out_layout=BFQ_SCALES_ROW_MAJOR, out_scale_ld=None, out_eps=DEFAULT_EPS,
                   preact=None, tile=None, workspace=None, workspace_bytes=None, stream=None,
                   w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32) -> int:
    """out[m][f] = act(g) * u, both factors block-scaled products of token row m (a_q [M, K]) with
    rows f and F + f of w_q [2F, K] (row-major or packed), w_scales [2F/128, K/128]. out [M, F]
    bf16 / fp16 / fp32, or e4m3fn codes (uint8 / float8_e4m3fn) with out_scales, one per 128
    columns, in out_layout. preact: bf16 [M, 2F] that receives (g, u)."""
    M, K = _shape2(a_q, "a_q")
    rows = _shape2(w_q, "w_q")[0]
    if rows % 2 != 0:
        raise BfqArgumentError(f"w_q has {rows} rows; expected the gate rows and as many up rows")
    F = rows // 2
    _rows(a_q, "a_q", U8_CODES, M, K)
    _rows(w_q, "w_q", U8_CODES, 2 * F, K)
    if a_scale_ld is None:
        a_scale_ld = a_scales.stride(0)
    _scales(a_scales, "a_scales", a_layout, a_scale_ld, M, K // 128, write=False)
    _flat(w_scales, "w_scales", ("float32",), (2 * F // 128) * (K // 128))
    _rows(out, "out", OUT_DTYPES + U8_CODES, M, F)
    codes = not isinstance(out, int) and _dt(out) in U8_CODES
    if codes != (out_scales is not None):
        raise BfqArgumentError("out_scales goes with an out of codes, and only with it")
    if codes:
        if out_scale_ld is None:
            out_scale_ld = out_scales.stride(0)
        _scales(out_scales, "out_scales", out_layout, out_scale_ld, M, F // 128, write=True)
    if preact is not None:
        _rows(preact, "preact", ("bfloat16",), M, 2 * F)
    workspace_bytes = _workspace_arg(workspace, workspace_bytes)
    _workspace(workspace, workspace_bytes)
    _devices(a_q=a_q, a_scales=a_scales, w_q=w_q, w_scales=w_scales, out=out,
             out_scales=out_scales, preact=preact, workspace=workspace)
    st = lib.bfq_gated_gemm(_ptr(a_q), _ptr(a_scales), a_layout, a_scale_ld, _ptr(w_q),
                            _ptr(w_scales), w_layout, scale_fmt, act, _ptr(out), _ptr(out_scales),
                            out_layout, out_scale_ld or 0, out_eps, _ptr(preact), M, F, K,
                            _block_shape(BLOCK_SHAPE), BFQ_E4M3FN,
                            BFQ_E4M3FN if codes else _odtype(out),
                            ctypes.byref(tile) if tile else None, _ptr(workspace),
                            workspace_bytes, _stream(stream))
    return _check(st, "bfq_gated_gemm")


def bfq_gated_backward(preact, dh, act=BFQ_ACT_SILU, dpre=None, q=None, scales=None,
                       layout=BFQ_SCALES_ROW_MAJOR, scale_ld=None, q_eps=DEFAULT_EPS,
                       scale_fmt=BFQ_SCALE_FP32, h=None, stream=None) -> int:
    """Gradient of act(g) * u at preact = (g, u) bf16 [M, 2F], for dh bf16 [M, F]: dpre bf16
    [M, 2F], and / or q (codes [M, 2F]) with scales (one per 128 columns); h bf16 [M, F] receives
    the product again."""
    M, F = _shape2(dh, "dh")
    _rows(preact, "preact", ("bfloat16",), M, 2 * F)
    _rows(dh, "dh", ("bfloat16",), M, F)
    if dpre is not None:
        _rows(dpre, "dpre", ("bfloat16",), M, 2 * F)
    if h is not None:
        _rows(h, "h", ("bfloat16",), M, F)
    if (q is None) != (scales is None):
        raise BfqArgumentError("q and scales go together")
    if q is not None:
        _rows(q, "q", CODE_DTYPES, M, 2 * F)
        if scale_ld is None:
            scale_ld = scales.stride(0)
        _scales(scales, "scales", layout, scale_ld, M, 2 * F // 128, write=True)
    _devices(preact=preact, dh=dh, dpre=dpre, q=q, scales=scales, h=h)
    st = lib.bfq_gated_backward(_ptr(preact), _ptr(dh), act, _ptr(dpre), _ptr(q),
                                _qdtype(q) if q is not None else BFQ_E4M3FN, _ptr(scales), layout,
                                scale_ld or 0, q_eps, scale_fmt, _ptr(h), M, F, _stream(stream))
    return _check(st, "bfq_gated_backward")


def bfq_transpose_weights(w_q, w_scales, wt_q, wt_scales, stream=None) -> int:
    """w_q: row-major codes [N, K] with w_scales [N/128, K/128]; wt_q [K, N] and wt_scales
    [K/128, N/128] receive the transpose (row-major)."""
    N, K = _shape2(w_q, "w_q")
    _rows(w_q, "w_q", CODE_DTYPES, N, K)
    _rows(wt_q, "wt_q", CODE_DTYPES, K, N)
    _same_codes(w_q, wt_q)
    _flat(w_scales, "w_scales", ("float32",), (N // 128) * (K // 128))
    _flat(wt_scales, "wt_scales", ("float32",), (N // 128) * (K // 128))
    _devices(w_q=w_q, w_scales=w_scales, wt_q=wt_q, wt_scales=wt_scales)
    st = lib.bfq_transpose_weights(_ptr(w_q), _ptr(w_scales), N, K, _qdtype(w_q), _ptr(wt_q),
                                   _ptr(wt_scales), _stream(stream))
    return _check(st, "bfq_transpose_weights")


RES_DTYPES = ("bfloat16", "float32")


def _norm_operands(residual, name, y, w_post, gate, gate_kind, w_pre):
    """Checks of what the norm step and its gradients share; returns (M, K, res_dtype)."""
    M, K = _shape2(residual, name)
    _rows(residual, name, RES_DTYPES, M, K)
    if y is not None:
        _rows(y, "y", ("bfloat16",), M, K)
    for n, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None:
            _flat(w, n, ("bfloat16",), K)
    if (gate is None) != (gate_kind == BFQ_GATE_NONE):
        raise BfqArgumentError("gate goes with a gate_kind other than BFQ_GATE_NONE, and only with it")
    if gate is not None:
        if gate_kind == BFQ_GATE_FULL:
            _rows(gate, "gate", ("bfloat16",), M, K)
        else:
            _flat(gate, "gate", ("bfloat16",), M if gate_kind == BFQ_GATE_TOKEN else K)
    return M, K, BFQ_BF16 if _dt(residual) == "bfloat16" else BFQ_FP32


def bfq_norm_residual(residual, y=None, w_post=None, gate=None, gate_kind=BFQ_GATE_NONE,
                      res_scale=1.0, w_pre=None, norm_eps=NORM_EPS, res_out=None, normed=None,
                      q=None, scales=None, layout=BFQ_SCALES_ROW_MAJOR, scale_ld=None,
                      q_eps=DEFAULT_EPS, group_size=128, scale_fmt=BFQ_SCALE_FP32,
                      stream=None) -> int:
    """One step of the residual stream: r' = residual + res_scale * gate * z with z = y or the
    RMS norm of y times w_post, stored in res_out (which may be residual); then the RMS norm of r'
    times w_pre, as normed (bf16 [M, K]) and / or codes q with scales. residual bf16 or fp32
    [M, K], y bf16 [M, K] or None, gate bf16 [K], [M] or [M, K] by gate_kind."""
    M, K, rt = _norm_operands(residual, "residual", y, w_post, gate, gate_kind, w_pre)
    if res_out is not None:
        _rows(res_out, "res_out", (_dt(residual),), M, K)
    if normed is not None:
        _rows(normed, "normed", ("bfloat16",), M, K)
    if (q is None) != (scales is None):
        raise BfqArgumentError("q and scales go together")
    if q is not None:
        _rows(q, "q", CODE_DTYPES, M, K)
        if scale_ld is None:
            scale_ld = scales.stride(0)
        if group_size > 0 and K % group_size == 0:
            _scales(scales, "scales", layout, scale_ld, M, K // group_size, write=True)
    _devices(residual=residual, y=y, w_post=w_post, gate=gate, w_pre=w_pre, res_out=res_out,
             normed=normed, q=q, scales=scales)
    st = lib.bfq_norm_residual(_ptr(y), _ptr(residual), rt, _ptr(w_post), _ptr(gate), gate_kind,
                               res_scale, _ptr(w_pre), norm_eps, _ptr(res_out), _ptr(normed),
                               _ptr(q), _qdtype(q) if q is not None else BFQ_E4M3FN, group_size,
                               _ptr(scales), layout, scale_ld or 0, q_eps, scale_fmt, M, K,
                               _stream(stream))
    return _check(st, "bfq_norm_residual")


def bfq_norm_residual_backward_workspace_bytes(M, K) -> int:
    return int(lib.bfq_norm_residual_backward_workspace_bytes(M, K))


def bfq_norm_residual_backward(res_out, d_res, y=None, w_post=None, gate=None,
                               gate_kind=BFQ_GATE_NONE, res_scale=1.0, w_pre=None,
                               norm_eps=NORM_EPS, d_normed=None, d_res_out=None, d_y=None,
                               d_w_pre=None, d_w_post=None, d_gate=None, workspace=None,
                               workspace_bytes=None, stream=None) -> int:
    """Gradients of bfq_norm_residual from the stored sum res_out, the gradient d_normed (bf16) of
    its normed output and d_res_out (res_out's dtype) of the sum: d_res (res_out's dtype; may be
    d_res_out), d_y (bf16), and where wanted d_w_pre, d_w_post (fp32 [K]) and d_gate (fp32 [K] or
    [M], bf16 [M, K] for a full gate)."""
    M, K, rt = _norm_operands(res_out, "res_out", y, w_post, gate, gate_kind, w_pre)
    _rows(d_res, "d_res", (_dt(res_out),), M, K)
    if d_res_out is not None:
        _rows(d_res_out, "d_res_out", (_dt(res_out),), M, K)
    for n, t in (("d_normed", d_normed), ("d_y", d_y)):
        if t is not None:
            _rows(t, n, ("bfloat16",), M, K)
    for n, t in (("d_w_pre", d_w_pre), ("d_w_post", d_w_post)):
        if t is not None:
            _flat(t, n, ("float32",), K)
    if d_gate is not None:
        if gate_kind == BFQ_GATE_FULL:
            _rows(d_gate, "d_gate", ("bfloat16",), M, K)
        else:
            _flat(d_gate, "d_gate", ("float32",), M if gate_kind == BFQ_GATE_TOKEN else K)
    workspace_bytes = _workspace_arg(workspace, workspace_bytes)
    _workspace(workspace, workspace_bytes)
    _devices(res_out=res_out, y=y, w_post=w_post, gate=gate, w_pre=w_pre, d_normed=d_normed,
             d_res_out=d_res_out, d_res=d_res, d_y=d_y, d_w_pre=d_w_pre, d_w_post=d_w_post,
             d_gate=d_gate, workspace=workspace)
    st = lib.bfq_norm_residual_backward(_ptr(y), _ptr(res_out), rt, _ptr(w_post), _ptr(gate),
                                        gate_kind, res_scale, _ptr(w_pre), norm_eps,
                                        _ptr(d_normed), _ptr(d_res_out), _ptr(d_res), _ptr(d_y),
                                        _ptr(d_w_pre), _ptr(d_w_post), _ptr(d_gate), M, K,
                                        _ptr(workspace), workspace_bytes, _stream(stream))
    return _check(st, "bfq_norm_residual_backward")


# ------------------------------------------------------------ allocating conveniences
#
# With `stream`, tensors are allocated under that stream, and outputs and operands are marked as used
# by both: the caching allocator orders a block's next use only behind the work of the stream that it
# was allocated under and of those it is told of, so a workspace from the caller's stream would be
# given out again while the launch still uses it. As with any work on a side stream, the caller orders
# the writes of the operands before the call and the use of the outputs after it.

def _side_stream(stream):
    """The torch stream of `stream` (a Stream or a raw handle) if it is not the current one."""
    torch = _torch or _torch_module()
    if not torch.cuda.is_initialized():          # no GPU tensor exists: the call is refused below
        return None
    handle = _stream(stream)
    if handle == _stream(None):
        return None
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _used_on(stream, values):
    for t in values:
        if isinstance(t, _Tensor):
            t.record_stream(stream)


def _under_stream(fn):
    """Runs an allocating convenience with its `stream` as torch's current one."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        side = None if stream is None else _side_stream(stream)
        if side is None:
            return fn(*args, **kw)
        caller = _torch.cuda.current_stream()
        with _torch.cuda.stream(side):
            out = fn(*args, **kw)
        # either may be dropped with the other stream's work on it in flight
        _used_on(side, (*args, *kw.values()))
        _used_on(caller, out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,))
        return out
    return call


@_under_stream
def quant_tokens(x, q_dtype=BFQ_E4M3FN, layout=BFQ_SCALES_ROW_MAJOR, eps=DEFAULT_EPS,
                 stream=None, scale_fmt=BFQ_SCALE_FP32, per_token=False):
    """Allocate (q, scales) with torch and run bfq_quant_tokens. Returns (q, scales); with
    per_token the scales are [M, 1] (row-major) or [1, M] (column-major); with
    BFQ_SCALES_PACKED_UE8M0 they are int32 words [ceil(K/512), round_up(M, 4)]."""
    import torch
    M, K = x.shape
    group = K if per_token else 128
    q = torch.empty((M, K), dtype=torch.uint8 if q_dtype == BFQ_E4M3FN else torch.int8,
                    device=x.device)
    if layout == BFQ_SCALES_ROW_MAJOR:
        s = torch.empty((M, K // group), dtype=torch.float32, device=x.device)
    elif layout == BFQ_SCALES_PACKED_UE8M0:     # int32 words [ceil(G/4), round_up(M, 4)]
        s = torch.empty(((K // 128 + 3) // 4, (M + 3) // 4 * 4), dtype=torch.int32,
                        device=x.device)
    else:
        s = torch.empty((K // group, M), dtype=torch.float32, device=x.device)
    bfq_quant_tokens(x, q, s, layout=layout, scale_ld=s.stride(0), eps=eps, stream=stream,
                     scale_fmt=scale_fmt, group_size=group)
    return q, s


@_under_stream
def quant_weight_blocks(w, q_dtype=BFQ_E4M3FN, eps=DEFAULT_EPS, stream=None,
                        scale_fmt=BFQ_SCALE_FP32, per_channel=False):
    """Allocate (q, scales) with torch and run bfq_quant_weight_blocks; per_channel gives one
    scale per output channel (scales [N])."""
    import torch
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8 if q_dtype == BFQ_E4M3FN else torch.int8,
                    device=w.device)
    if per_channel:
        s = torch.empty((N,), dtype=torch.float32, device=w.device)
        bs = channel_block_shape(K)
    else:
        s = torch.empty((N // 128, K // 128), dtype=torch.float32, device=w.device)
        bs = BLOCK_SHAPE
    bfq_quant_weight_blocks(w, q, s, eps=eps, stream=stream, scale_fmt=scale_fmt, block_shape=bs)
    return q, s


@_under_stream
def moe_align(topk_ids, E, stream=None):
    """Allocate and run bfq_moe_align. Returns (expert_offsets int32 [E+1], sorted_pairs
    int32 [T*topk])."""
    import torch
    T, topk = topk_ids.shape
    dev = topk_ids.device
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    srt = torch.empty(T * topk, dtype=torch.int32, device=dev)
    need = int(lib.bfq_moe_align_workspace_bytes(T, topk, E))
    ws = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    bfq_moe_align(topk_ids, E, off, srt, workspace=ws, stream=stream)
    return off, srt


@_under_stream
def moe_block_gemm(a_q, a_scales, sorted_pairs, expert_offsets, topk, w_q, w_scales,
                   out_dtype=None, a_layout=BFQ_SCALES_ROW_MAJOR, tile=None, stream=None,
                   w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32):
    """Allocate out [T*topk, N] (and split-K workspace) with torch and run bfq_moe_block_gemm."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    T, K = a_q.shape
    E, N = w_q.shape[0], w_q.shape[1]
    out = torch.empty((T * topk, N), dtype=out_dtype, device=a_q.device)
    if tile is None:
        st, tile = bfq_moe_select_tile(T, topk, E, N, K, _odtype(out), w_layout, scale_fmt)
        _check(st, "bfq_moe_select_tile", warn_key=("moe", E, N, K), depth=4)
    ws_bytes = bfq_moe_gemm_workspace_bytes(T, topk, N, tile)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=a_q.device) if ws_bytes else None
    bfq_moe_block_gemm(a_q, a_scales, sorted_pairs, expert_offsets, topk, w_q, w_scales, out,
                       a_layout=a_layout, tile=tile, workspace=ws, workspace_bytes=ws_bytes,
                       stream=stream, w_layout=w_layout, scale_fmt=scale_fmt)
    return out


@_under_stream
def pack_weights(w_q, stream=None):
    """Allocate a packed copy of row-major weight codes (same dtype and shape) with torch and
    run bfq_pack_weights. [E, N, K] expert weights pack as one [E*N, K] matrix, which is each
    expert packed in turn (16-row fragments never straddle experts, N being a multiple of
    128)."""
    import torch
    p = torch.empty_like(w_q, memory_format=torch.contiguous_format)
    bfq_pack_weights(w_q.reshape(-1, w_q.shape[-1]), p.view(-1, w_q.shape[-1]), stream=stream)
    return p


@_under_stream
def block_gemm(a_q, a_scales, w_q, w_scales, out_dtype=None, a_layout=BFQ_SCALES_ROW_MAJOR,
               tile=None, stream=None, w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32,
               per_channel=False):
    """Allocate out (and split-K workspace) with torch and run bfq_block_gemm; per_channel
    selects the per-token x per-channel format (block_shape (1, K))."""
    import torch
    out_dtype = out_dtype or torch.bfloat16
    M, K = a_q.shape
    N = w_q.shape[0]
    bs = channel_block_shape(K) if per_channel else BLOCK_SHAPE
    out = torch.empty((M, N), dtype=out_dtype, device=a_q.device)
    if tile is None:
        st, tile = bfq_select_tile(M, N, K, _qdtype(a_q), _odtype(out), w_layout=w_layout,
                                   scale_fmt=scale_fmt, block_shape=bs)
        _check(st, "bfq_select_tile", warn_key=(N, K), depth=4)
    ws_bytes = bfq_gemm_workspace_bytes(M, N, K, tile)
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=a_q.device) if ws_bytes else None
    bfq_block_gemm(a_q, a_scales, w_q, w_scales, out, a_layout=a_layout, tile=tile,
                   workspace=ws, workspace_bytes=ws_bytes, stream=stream, w_layout=w_layout,
                   scale_fmt=scale_fmt, block_shape=bs)
    return out


def _alloc_scales(M, groups, layout, device):
    """An empty scale tensor of the quantizers' output in `layout`."""
    import torch
    if layout == BFQ_SCALES_PACKED_UE8M0:
        return torch.empty(((groups + 3) // 4, (M + 3) // 4 * 4), dtype=torch.int32, device=device)
    shape = (M, groups) if layout == BFQ_SCALES_ROW_MAJOR else (groups, M)
    return torch.empty(shape, dtype=torch.float32, device=device)


@_under_stream
def gated_gemm(a_q, a_scales, w_q, w_scales, act=BFQ_ACT_SILU, out_dtype=None, codes=False,
               keep_preact=False, a_layout=BFQ_SCALES_ROW_MAJOR, out_layout=BFQ_SCALES_ROW_MAJOR,
               tile=None, stream=None, w_layout=BFQ_W_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32):
    """Allocate and run bfq_gated_gemm. Returns out, or (codes, scales) with `codes`; with
    keep_preact followed by the bf16 pre-activations [M, 2F]."""
    import torch
    M, K = a_q.shape
    F, dev = w_q.shape[0] // 2, a_q.device
    out = torch.empty((M, F), dtype=torch.uint8 if codes else out_dtype or torch.bfloat16, device=dev)
    scales = _alloc_scales(M, F // 128, out_layout, dev) if codes else None
    pre = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if keep_preact else None
    n = bfq_gated_gemm_workspace_bytes(M, F, K, BFQ_E4M3FN if codes else _odtype(out), w_layout,
                                       scale_fmt, tile)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    bfq_gated_gemm(a_q, a_scales, w_q, w_scales, out, act=act, a_layout=a_layout,
                   out_scales=scales, out_layout=out_layout, preact=pre, tile=tile, workspace=ws,
                   stream=stream, w_layout=w_layout, scale_fmt=scale_fmt)
    res = ((out, scales) if codes else (out,)) + ((pre,) if keep_preact else ())
    return res if len(res) > 1 else out


@_under_stream
def gated_backward(preact, dh, act=BFQ_ACT_SILU, codes=False, want_h=False,
                   layout=BFQ_SCALES_ROW_MAJOR, q_dtype=BFQ_E4M3FN, scale_fmt=BFQ_SCALE_FP32,
                   stream=None):
    """Allocate and run bfq_gated_backward. Returns dpre (bf16), or (codes, scales) with `codes`;
    with want_h followed by the product act(g) * u."""
    import torch
    M, F = dh.shape
    dev = dh.device
    q = scales = dpre = None
    if codes:
        q = torch.empty((M, 2 * F), dtype=torch.uint8 if q_dtype == BFQ_E4M3FN else torch.int8,
                        device=dev)
        scales = _alloc_scales(M, 2 * F // 128, layout, dev)
    else:
        dpre = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev)
    h = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if want_h else None
    bfq_gated_backward(preact, dh, act=act, dpre=dpre, q=q, scales=scales, layout=layout,
                       scale_fmt=scale_fmt, h=h, stream=stream)
    res = ((q, scales) if codes else (dpre,)) + ((h,) if want_h else ())
    return res if len(res) > 1 else dpre


@_under_stream
def transpose_weights(w_q, w_scales, stream=None):
    """Allocate and run bfq_transpose_weights: (codes [K, N], scales [K/128, N/128])."""
    import torch
    N, K = w_q.shape
    wt = torch.empty((K, N), dtype=w_q.dtype, device=w_q.device)
    st = torch.empty((K // 128, N // 128), dtype=torch.float32, device=w_q.device)
    bfq_transpose_weights(w_q, w_scales, wt, st, stream=stream)
    return wt, st


@_under_stream
def norm_residual(residual, y=None, w_post=None, gate=None, gate_kind=BFQ_GATE_NONE, res_scale=1.0,
                  w_pre=None, norm_eps=NORM_EPS, codes=False, q_dtype=BFQ_E4M3FN, per_token=False,
                  layout=BFQ_SCALES_ROW_MAJOR, scale_fmt=BFQ_SCALE_FP32, stream=None):
    """Allocate and run bfq_norm_residual. Returns a tuple: the new residual (with y), then (with
    w_pre) the normed bf16 rows or, with `codes`, their codes and scales."""
    import torch
    M, K = residual.shape
    dev = residual.device
    res_out = torch.empty_like(residual) if y is not None else None
    q = scales = normed = None
    group = K if per_token else 128
    if w_pre is not None and codes:
        q = torch.empty((M, K), dtype=torch.uint8 if q_dtype == BFQ_E4M3FN else torch.int8, device=dev)
        scales = _alloc_scales(M, K // group, layout, dev)
    elif w_pre is not None:
        normed = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    bfq_norm_residual(residual, y=y, w_post=w_post, gate=gate, gate_kind=gate_kind,
                      res_scale=res_scale, w_pre=w_pre, norm_eps=norm_eps, res_out=res_out,
                      normed=normed, q=q, scales=scales, layout=layout, group_size=group,
                      scale_fmt=scale_fmt, stream=stream)
    return tuple(t for t in (res_out, normed, q, scales) if t is not None)


@_under_stream
def norm_residual_backward(res_out, y=None, w_post=None, gate=None, gate_kind=BFQ_GATE_NONE,
                           res_scale=1.0, w_pre=None, norm_eps=NORM_EPS, d_normed=None,
                           d_res_out=None, stream=None) -> dict:
    """Allocate and run bfq_norm_residual_backward for every gradient its operands have. Returns
    {"d_res", "d_y", "d_w_pre", "d_w_post", "d_gate"}, without those whose operand is absent."""
    import torch
    M, K = res_out.shape
    dev = res_out.device
    g = {"d_res": torch.empty_like(res_out)}
    if y is not None:
        g["d_y"] = torch.empty_like(y)
    for n, w in (("d_w_pre", w_pre), ("d_w_post", w_post)):
        if w is not None:
            g[n] = torch.empty(K, dtype=torch.float32, device=dev)
    if gate is not None:
        g["d_gate"] = torch.empty(gate.shape, device=dev,
                                  dtype=torch.bfloat16 if gate_kind == BFQ_GATE_FULL else torch.float32)
    n = bfq_norm_residual_backward_workspace_bytes(M, K)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    bfq_norm_residual_backward(res_out, y=y, w_post=w_post, gate=gate, gate_kind=gate_kind,
                               res_scale=res_scale, w_pre=w_pre, norm_eps=norm_eps,
                               d_normed=d_normed, d_res_out=d_res_out, workspace=ws, stream=stream,
                               **g)
    return g
