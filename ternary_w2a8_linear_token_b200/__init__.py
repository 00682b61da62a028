"""Python binding of libbitnet (the B200 W2A8 BitLinear library).

Argument marshalling only: every step of the forward runs in the CUDA kernels behind
the C ABI declared in ``include/bitnet.h``. PyTorch supplies device memory (output and
workspace tensors) and the current CUDA stream; nothing here computes on tensors.

The shared library is built in-tree by ``python ternary_w2a8_linear_token_b200/build.py``.
Importing this package without it raises ImportError: there is no fallback path.

Functions keep the C names:
    bitnet_pack_weights(W, per_row)            -> (packed, s_w)
    bitnet_pack_ternary(t)                     -> packed
    bitnet_quant_act(x)                        -> (q, s_x)
    bitnet_linear(x, packed, s_w, per_row, ...) -> y
    bitnet_linear_batch(x, projs, ...)         -> [y, ...]
    bitnet_linear_i32(q, packed, ...)          -> acc (int32)
    bitnet_interleave_gate_up(pg, sg, pu, su, per_row) -> (packed_gu, s_w_gu)
    bitnet_linear_swiglu(x, packed_gu, s_w_gu, per_row, ...) -> h (bf16)
    bitnet_pack_w4(W, group)                   -> (packed, scales)
    bitnet_linear_w4(x, packed, scales, group, ...) -> y
    bitnet_cache_fork / _extend / _free / _compact / _copy / _append(cache, ...)
    bitnet_paged_attention(q, cache, layer, ...) -> out or (out, lse)
    bitnet_check_device_errors()               -> watchdog word (0 = clean)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbitnet.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python ternary_w2a8_linear_token_b200/build.py` "
        "(there is no non-CUDA fallback)")

lib = ctypes.CDLL(LIB_PATH)

# ----------------------------------------------------------------------------- constants
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(8)
SCALE_PER_TENSOR, SCALE_PER_ROW = 0, 1
OUT_BF16, OUT_F32 = 0, 1
PATH_AUTO, PATH_GEMV, PATH_TC, PATH_MMA = 0, 1, 2, 3
ACT_PER_TOKEN, ACT_PER_TENSOR = 0, 1
QUANT_WORKSPACE_BYTES = 4096
GEMV_MAX_M = 8
GEMV_AUTO_M = 4  # PATH_AUTO: GEMV up to here; 5..8 tokens take the tensor-core path given a workspace
WATCHDOG_TMA_FULL, WATCHDOG_UNPACK, WATCHDOG_EMPTY, WATCHDOG_ACCUM, WATCHDOG_DRAIN = (
    1 << 0, 1 << 1, 1 << 2, 1 << 3, 1 << 4)
WATCHDOG_SELFTEST = 1 << 6
MAX_PROJ = 8
CACHE_BF16, CACHE_I8 = 0, 1
CACHE_ERR_SEQ, CACHE_ERR_LEN, CACHE_ERR_PAGE, CACHE_ERR_FULL = 1 << 0, 1 << 1, 1 << 2, 1 << 3
CACHE_MAX_LAYERS = 64
SWIGLU_BLOCK = 16  # interleaved gate/up rows come in blocks of this many

_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t


class bitnet_proj(ctypes.Structure):
    _fields_ = [("packed", _P), ("s_w", _P), ("mode", _I32), ("reserved", _I32), ("N", _I64),
                ("y", _P)]


class bitnet_plan(ctypes.Structure):
    _fields_ = [("kernel", _I32), ("grid", _I32), ("tile_tokens", _I32), ("splits", _I32),
                ("tile_rows", _I32), ("reserved", _I32 * 3)]


class bitnet_cache(ctypes.Structure):
    _fields_ = [("table", _P), ("lens", _P), ("refs", _P), ("error", _P), ("num_pages", _I64),
                ("max_seqs", _I64), ("max_pages", _I64), ("page_size", _I32), ("kv_heads", _I32),
                ("head_dim", _I32), ("dtype", _I32)]


class bitnet_cache_layer(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P)]


KERNEL_GEMV, KERNEL_MMA_GEMV, KERNEL_STREAM, KERNEL_TC, KERNEL_GS = 1, 2, 3, 4, 5

_SIGS = {
    "bitnet_pack_weights": ([_P, _I64, _I64, ctypes.c_int, _P, _P, _P], ctypes.c_int),
    "bitnet_pack_ternary": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "bitnet_quant_act": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "bitnet_linear_workspace_size": ([_I64, _I64], _SZ),
    "bitnet_quant_act_ex": ([_P, _I64, _I64, ctypes.c_int, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "bitnet_linear_batch_act": ([_P, _I64, _I64, ctypes.POINTER(bitnet_proj), _I32, ctypes.c_int,
                                 ctypes.c_int, _P, _SZ, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_linear": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _P, _SZ, _P],
                      ctypes.c_int),
    "bitnet_linear_ex": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _P, _SZ,
                          ctypes.c_int, _P], ctypes.c_int),
    "bitnet_linear_batch": ([_P, _I64, _I64, ctypes.POINTER(bitnet_proj), _I32, ctypes.c_int, _P,
                             _SZ, _P], ctypes.c_int),
    "bitnet_linear_batch_ex": ([_P, _I64, _I64, ctypes.POINTER(bitnet_proj), _I32, ctypes.c_int,
                                _P, _SZ, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_linear_i32": ([_P, _I64, _I64, _P, _I64, _P, _P, _SZ, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_linear_noalloc": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _P],
                              ctypes.c_int),
    "bitnet_interleave_gate_up": ([_P, _P, _P, _P, ctypes.c_int, _I64, _I64, _P, _P, _P],
                                  ctypes.c_int),
    "bitnet_linear_swiglu": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, _P, _SZ,
                             ctypes.c_int, _P], ctypes.c_int),
    "bitnet_linear_swiglu_hmax": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, _P, _P, _SZ,
                                   _P], ctypes.c_int),
    "bitnet_linear_hmax": ([_P, _P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _P,
                            _SZ, _P], ctypes.c_int),
    "bitnet_quant_act_hmax": ([_P, _P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "bitnet_b3_row_bytes": ([_I64], _I64),
    "bitnet_pack_ternary_b3": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "bitnet_linear_b3": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _P],
                         ctypes.c_int),
    "bitnet_act_amax": ([_P, _I64, _I64, _P, _P], ctypes.c_int),
    "bitnet_quant_act_amax": ([_P, _I64, _I64, _P, _P, _P, _P], ctypes.c_int),
    "bitnet_dequant": ([_P, _I64, _I64, _P, _P, ctypes.c_int, _P, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_linear_plan": ([_I64, _I64, ctypes.POINTER(_I64), _I32, _I32, _SZ, ctypes.c_int,
                            ctypes.POINTER(bitnet_plan)], ctypes.c_int),
    "bitnet_w4_row_bytes": ([_I64], _I64),
    "bitnet_pack_w4": ([_P, _I64, _I64, _I32, _P, _P, _P], ctypes.c_int),
    "bitnet_linear_w4": ([_P, _I64, _I64, _P, _P, _I32, _I64, _P, ctypes.c_int, _P], ctypes.c_int),
    "bitnet_cache_workspace_size": ([ctypes.POINTER(bitnet_cache), _I64], _SZ),
    "bitnet_cache_fork": ([ctypes.POINTER(bitnet_cache), _P, _P, _I64, _P, _SZ, _P], ctypes.c_int),
    "bitnet_cache_extend": ([ctypes.POINTER(bitnet_cache), _P, _P, _I64, _P, _I64, _P, _SZ, _P],
                            ctypes.c_int),
    "bitnet_cache_free": ([ctypes.POINTER(bitnet_cache), _P, _I64, _P, _SZ, _P], ctypes.c_int),
    "bitnet_cache_compact": ([ctypes.POINTER(bitnet_cache), _P, _I64, _P, _SZ, _P], ctypes.c_int),
    "bitnet_cache_copy": ([ctypes.POINTER(bitnet_cache), ctypes.POINTER(bitnet_cache_layer), _I32,
                           _P, _I64, _P], ctypes.c_int),
    "bitnet_cache_append": ([ctypes.POINTER(bitnet_cache), ctypes.POINTER(bitnet_cache_layer), _P,
                             _P, _I64, _P, _P, _P], ctypes.c_int),
    "bitnet_paged_attention_workspace_size": ([ctypes.POINTER(bitnet_cache), _I64, _I64], _SZ),
    "bitnet_paged_attention": ([ctypes.POINTER(bitnet_cache), ctypes.POINTER(bitnet_cache_layer),
                                _P, _I64, _I64, _P, ctypes.c_float, _I64, _I64, _P, _P, _P, _SZ,
                                _P], ctypes.c_int),
    "bitnet_check_device_errors": ([ctypes.POINTER(_I32)], ctypes.c_int),
    "bitnet_selftest_wait_timeout": ([_I64, _P], ctypes.c_int),
    "bitnet_probe_int_rate": ([_I32, _I32, _I64, _P, _P], ctypes.c_int),
    "bitnet_probe_int_ops": ([_I32, _I32, _I64], _I64),
    "bitnet_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "bitnet_version": ([], _I32),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class BitnetError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.bitnet_status_string(status).decode()} ({status})")


def _check(status: int, where: str):
    if status != OK:
        raise BitnetError(status, where)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _x_ptr(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return _dev(x, torch.bfloat16, "x")
    return _dev(x, torch.int16, "x (bf16 bits)")


def _check_proj(packed: torch.Tensor, s_w: torch.Tensor, per_row: bool, K: int,
                name: str = "packed") -> int:
    """Shape checks the C side cannot make (it sees only pointers): packed (N, K/4) and s_w
    of N (per row) or 1 (per tensor) elements. Returns N."""
    if packed.dim() != 2 or packed.shape[1] * 4 != K:
        raise ValueError(f"{name} must be (N, K/4) = (N, {K // 4}), got {tuple(packed.shape)}")
    N = packed.shape[0]
    want = N if per_row else 1
    if s_w.numel() != want:
        raise ValueError(f"s_w must have {want} element(s) ({'per row' if per_row else 'per tensor'})"
                         f", got {s_w.numel()}")
    return N


def _check_out(y: torch.Tensor, M: int, N: int, name: str = "y"):
    if tuple(y.shape) != (M, N):
        raise ValueError(f"{name} must be ({M}, {N}), got {tuple(y.shape)}")
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} must be bfloat16 or float32, got {y.dtype}")


def workspace_size(M: int, K: int) -> int:
    return int(lib.bitnet_linear_workspace_size(M, K))


def make_workspace(M: int, K: int, device=None) -> torch.Tensor:
    """A device buffer big enough for the tensor-core path at (M, K) (256-byte aligned)."""
    n = workspace_size(M, K)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


# ----------------------------------------------------------------------------- calls
def bitnet_pack_weights(W: torch.Tensor, per_row: bool, stream=None):
    N, K = W.shape
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    s_w = torch.empty(N if per_row else 1, dtype=torch.float32, device=W.device)
    _check(lib.bitnet_pack_weights(_dev(W, torch.float32, "W"), N, K, int(bool(per_row)),
                                   packed.data_ptr(), s_w.data_ptr(), _stream(stream)),
           "bitnet_pack_weights")
    return packed, s_w


def bitnet_pack_ternary(t: torch.Tensor, stream=None) -> torch.Tensor:
    N, K = t.shape
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=t.device)
    _check(lib.bitnet_pack_ternary(_dev(t, torch.int8, "t"), N, K, packed.data_ptr(),
                                   _stream(stream)), "bitnet_pack_ternary")
    return packed


def bitnet_quant_act(x: torch.Tensor, stream=None):
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s_x = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitnet_quant_act(_x_ptr(x), M, K, q.data_ptr(), s_x.data_ptr(), _stream(stream)),
           "bitnet_quant_act")
    return q, s_x


def bitnet_quant_act_ex(x: torch.Tensor, act: int = ACT_PER_TOKEN, stream=None):
    """bitnet_quant_act with a choice of scale granularity (ACT_PER_TOKEN / ACT_PER_TENSOR)."""
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s_x = torch.empty(M, dtype=torch.float32, device=x.device)
    ws = torch.empty(QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=x.device)
    _check(lib.bitnet_quant_act_ex(_x_ptr(x), M, K, act, q.data_ptr(), s_x.data_ptr(),
                                   ws.data_ptr(), ws.numel(), _stream(stream)),
           "bitnet_quant_act_ex")
    return q, s_x


@functools.lru_cache(maxsize=4096)
def _takes_tc_path(M: int, K: int, path: int) -> bool:
    """Whether a call of this shape runs the tensor-core path (and so needs a workspace): the
    library's own plan query, which also covers rows too long for the GEMV."""
    if path == PATH_TC:
        return True
    if path != PATH_AUTO:
        return False
    pl = bitnet_plan()
    arr = (_I64 * 1)(64)
    st = lib.bitnet_linear_plan(M, K, arr, 1, 0, workspace_size(M, K), path, ctypes.byref(pl))
    return st == OK and pl.kernel == KERNEL_TC


def _ws_args(workspace: Optional[torch.Tensor], M: int, K: int, path: int, device):
    if workspace is None:
        if not _takes_tc_path(M, K, path):
            return None, 0, None
        workspace = make_workspace(M, K, device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def bitnet_linear(x: torch.Tensor, packed: torch.Tensor, s_w: torch.Tensor, per_row: bool,
                  out_dtype: torch.dtype = torch.bfloat16, y: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, path: int = PATH_AUTO, stream=None):
    M, K = x.shape
    N = _check_proj(packed, s_w, per_row, K)
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check_out(y, M, N)
    od = OUT_BF16 if y.dtype == torch.bfloat16 else OUT_F32
    wp, wb, _keep = _ws_args(workspace, M, K, path, x.device)
    _check(lib.bitnet_linear_ex(_x_ptr(x), M, K, _dev(packed, torch.uint8, "packed"),
                                _dev(s_w, torch.float32, "s_w"), int(bool(per_row)), N,
                                _dev(y, y.dtype, "y"), od, wp, wb, path, _stream(stream)),
           "bitnet_linear")
    return y


def bitnet_linear_batch(x: torch.Tensor, projs: Sequence, out_dtype: torch.dtype = torch.bfloat16,
                        ys: Optional[Sequence[torch.Tensor]] = None,
                        workspace: Optional[torch.Tensor] = None, path: int = PATH_AUTO,
                        stream=None):
    """projs: sequence of (packed, s_w, per_row). Returns the list of outputs (M, N_i)."""
    M, K = x.shape
    n = len(projs)
    if not 1 <= n <= MAX_PROJ:
        raise ValueError(f"1..{MAX_PROJ} projections")
    Ns = [_check_proj(p[0], p[1], p[2], K) for p in projs]
    if ys is None:
        ys = [torch.empty((M, N), dtype=out_dtype, device=x.device) for N in Ns]
    if len(ys) != n:
        raise ValueError(f"{n} projections need {n} outputs, got {len(ys)}")
    for yi, N in zip(ys, Ns):
        _check_out(yi, M, N)
    if any(yi.dtype != ys[0].dtype for yi in ys):
        raise ValueError("all outputs of a batch must have one dtype")
    od = OUT_BF16 if ys[0].dtype == torch.bfloat16 else OUT_F32
    arr = (bitnet_proj * n)()
    for i, (packed, s_w, per_row) in enumerate(projs):
        arr[i].packed = _dev(packed, torch.uint8, "packed")
        arr[i].s_w = _dev(s_w, torch.float32, "s_w")
        arr[i].mode = int(bool(per_row))
        arr[i].reserved = 0
        arr[i].N = packed.shape[0]
        arr[i].y = _dev(ys[i], ys[i].dtype, "y")
    wp, wb, _keep = _ws_args(workspace, M, K, path, x.device)
    _check(lib.bitnet_linear_batch_ex(_x_ptr(x), M, K, arr, n, od, wp, wb, path, _stream(stream)),
           "bitnet_linear_batch")
    return list(ys)


def bitnet_linear_batch_act(x: torch.Tensor, projs: Sequence, act: int,
                            out_dtype: torch.dtype = torch.bfloat16,
                            ys: Optional[Sequence[torch.Tensor]] = None,
                            workspace: Optional[torch.Tensor] = None, path: int = PATH_AUTO,
                            stream=None):
    """bitnet_linear_batch with a choice of activation scale granularity (act)."""
    M, K = x.shape
    n = len(projs)
    if not 1 <= n <= MAX_PROJ:
        raise ValueError(f"1..{MAX_PROJ} projections")
    Ns = [_check_proj(p[0], p[1], p[2], K) for p in projs]
    if ys is None:
        ys = [torch.empty((M, N), dtype=out_dtype, device=x.device) for N in Ns]
    if len(ys) != n:
        raise ValueError(f"{n} projections need {n} outputs, got {len(ys)}")
    for yi, N in zip(ys, Ns):
        _check_out(yi, M, N)
    if any(yi.dtype != ys[0].dtype for yi in ys):
        raise ValueError("all outputs of a batch must have one dtype")
    od = OUT_BF16 if ys[0].dtype == torch.bfloat16 else OUT_F32
    arr = (bitnet_proj * n)()
    for i, (packed, s_w, per_row) in enumerate(projs):
        arr[i].packed = _dev(packed, torch.uint8, "packed")
        arr[i].s_w = _dev(s_w, torch.float32, "s_w")
        arr[i].mode = int(bool(per_row))
        arr[i].reserved = 0
        arr[i].N = packed.shape[0]
        arr[i].y = _dev(ys[i], ys[i].dtype, "y")
    wp, wb, _keep = _ws_args(workspace, M, K, path, x.device)
    _check(lib.bitnet_linear_batch_act(_x_ptr(x), M, K, arr, n, od, act, wp, wb, path,
                                       _stream(stream)), "bitnet_linear_batch_act")
    return list(ys)


def bitnet_linear_i32(q: torch.Tensor, packed: torch.Tensor, path: int = PATH_AUTO,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M, K = q.shape
    if packed.dim() != 2 or packed.shape[1] * 4 != K:
        raise ValueError(f"packed must be (N, K/4) = (N, {K // 4}), got {tuple(packed.shape)}")
    N = packed.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=q.device)
    wp, wb, _keep = _ws_args(workspace, M, K, path, q.device)
    _check(lib.bitnet_linear_i32(_dev(q, torch.int8, "q"), M, K,
                                 _dev(packed, torch.uint8, "packed"), N, acc.data_ptr(), wp, wb,
                                 path, _stream(stream)), "bitnet_linear_i32")
    return acc


def bitnet_interleave_gate_up(packed_gate: torch.Tensor, s_w_gate: torch.Tensor,
                              packed_up: torch.Tensor, s_w_up: torch.Tensor, per_row: bool,
                              stream=None):
    """Gate and up projections (each (I, K/4) packed) -> the interleaved (2I, K/4) matrix
    and its scales (2I per row, or {s_gate, s_up}) that bitnet_linear_swiglu reads."""
    I, K4 = packed_gate.shape
    if tuple(packed_up.shape) != (I, K4):
        raise ValueError("gate and up must have the same shape")
    dev = packed_gate.device
    packed_gu = torch.empty((2 * I, K4), dtype=torch.uint8, device=dev)
    s_w_gu = torch.empty(2 * I if per_row else 2, dtype=torch.float32, device=dev)
    _check(lib.bitnet_interleave_gate_up(_dev(packed_gate, torch.uint8, "packed_gate"),
                                         _dev(s_w_gate, torch.float32, "s_w_gate"),
                                         _dev(packed_up, torch.uint8, "packed_up"),
                                         _dev(s_w_up, torch.float32, "s_w_up"),
                                         int(bool(per_row)), I, 4 * K4, packed_gu.data_ptr(),
                                         s_w_gu.data_ptr(), _stream(stream)),
           "bitnet_interleave_gate_up")
    return packed_gu, s_w_gu


def bitnet_linear_swiglu(x: torch.Tensor, packed_gu: torch.Tensor, s_w_gu: torch.Tensor,
                         per_row: bool, h: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, path: int = PATH_AUTO,
                         stream=None) -> torch.Tensor:
    """h = bf16(bf16(silu(gate(x))) * up(x)), (M, I), from the interleaved gate/up matrix."""
    M, K = x.shape
    if packed_gu.dim() != 2 or packed_gu.shape[1] * 4 != K or packed_gu.shape[0] % 2:
        raise ValueError(f"packed_gu must be (2I, K/4) = (2I, {K // 4}), got "
                         f"{tuple(packed_gu.shape)}")
    I = packed_gu.shape[0] // 2
    want = 2 * I if per_row else 2
    if s_w_gu.numel() != want:
        raise ValueError(f"s_w_gu must have {want} elements, got {s_w_gu.numel()}")
    if h is None:
        h = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    if tuple(h.shape) != (M, I):
        raise ValueError(f"h must be ({M}, {I}), got {tuple(h.shape)}")
    wp, wb, _keep = _ws_args(workspace, M, K, path, x.device)
    _check(lib.bitnet_linear_swiglu(_x_ptr(x), M, K, _dev(packed_gu, torch.uint8, "packed_gu"),
                                    _dev(s_w_gu, torch.float32, "s_w_gu"), int(bool(per_row)), I,
                                    _dev(h, torch.bfloat16, "h"), wp, wb, path, _stream(stream)),
           "bitnet_linear_swiglu")
    return h


def _check_xmax(xmax: torch.Tensor, M: int, K: int):
    if tuple(xmax.shape) != (M, K // SWIGLU_BLOCK) or not xmax.is_contiguous():
        raise ValueError(f"xmax must be contiguous ({M}, {K // SWIGLU_BLOCK}), got "
                         f"{tuple(xmax.shape)}")
    return _dev(xmax, torch.int16, "xmax")


def bitnet_linear_swiglu_hmax(x: torch.Tensor, packed_gu: torch.Tensor, s_w_gu: torch.Tensor,
                              per_row: bool, h: Optional[torch.Tensor] = None,
                              hmax: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None):
    """bitnet_linear_swiglu on the tensor-core path that also returns hmax (M, I/16) int16:
    the bf16 bits of max |h| over each block of 16 outputs, for bitnet_linear_hmax."""
    M, K = x.shape
    if packed_gu.dim() != 2 or packed_gu.shape[1] * 4 != K or packed_gu.shape[0] % 2:
        raise ValueError(f"packed_gu must be (2I, K/4) = (2I, {K // 4}), got "
                         f"{tuple(packed_gu.shape)}")
    I = packed_gu.shape[0] // 2
    want = 2 * I if per_row else 2
    if s_w_gu.numel() != want:
        raise ValueError(f"s_w_gu must have {want} elements, got {s_w_gu.numel()}")
    if h is None:
        h = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    if hmax is None:
        hmax = torch.empty((M, I // SWIGLU_BLOCK), dtype=torch.int16, device=x.device)
    if tuple(h.shape) != (M, I):
        raise ValueError(f"h must be ({M}, {I}), got {tuple(h.shape)}")
    hm = _check_xmax(hmax, M, I)
    wp, wb, _keep = _ws_args(workspace, M, K, PATH_TC, x.device)
    _check(lib.bitnet_linear_swiglu_hmax(_x_ptr(x), M, K, _dev(packed_gu, torch.uint8, "packed_gu"),
                                         _dev(s_w_gu, torch.float32, "s_w_gu"),
                                         int(bool(per_row)), I, _dev(h, torch.bfloat16, "h"),
                                         hm, wp, wb, _stream(stream)),
           "bitnet_linear_swiglu_hmax")
    return h, hmax


def bitnet_linear_hmax(x: torch.Tensor, xmax: torch.Tensor, packed: torch.Tensor,
                       s_w: torch.Tensor, per_row: bool, out_dtype: torch.dtype = torch.bfloat16,
                       y: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """bitnet_linear on the tensor-core path with each token's amax taken from xmax, the
    (M, K/16) block maxima of |x| (as bitnet_linear_swiglu_hmax returns them for h)."""
    M, K = x.shape
    N = _check_proj(packed, s_w, per_row, K)
    xm = _check_xmax(xmax, M, K)
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check_out(y, M, N)
    od = OUT_BF16 if y.dtype == torch.bfloat16 else OUT_F32
    wp, wb, _keep = _ws_args(workspace, M, K, PATH_TC, x.device)
    _check(lib.bitnet_linear_hmax(_x_ptr(x), xm, M, K, _dev(packed, torch.uint8, "packed"),
                                  _dev(s_w, torch.float32, "s_w"), int(bool(per_row)), N,
                                  _dev(y, y.dtype, "y"), od, wp, wb, _stream(stream)),
           "bitnet_linear_hmax")
    return y


def bitnet_quant_act_hmax(x: torch.Tensor, xmax: torch.Tensor, stream=None):
    """bitnet_quant_act with each token's amax taken from xmax (M, K/16)."""
    M, K = x.shape
    xm = _check_xmax(xmax, M, K)
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s_x = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitnet_quant_act_hmax(_x_ptr(x), xm, M, K, q.data_ptr(), s_x.data_ptr(),
                                     _stream(stream)), "bitnet_quant_act_hmax")
    return q, s_x


NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def bitnet_linear_noalloc(x: torch.Tensor, packed: torch.Tensor, s_w: torch.Tensor,
                          per_row: bool, out_dtype: torch.dtype = torch.bfloat16,
                          y: Optional[torch.Tensor] = None, stream=None):
    """bitnet_linear without a workspace, for callers that cannot allocate device memory
    while they run (a serving loop where cudaMalloc could synchronise the device, a plug-in
    whose host runtime owns all device memory). The tensor-core path uses the library's
    fixed 16 MiB device scratch array; calls that can overlap on the GPU race on it. Sizes
    whose workspace exceeds the array raise BitnetError (ERR_WORKSPACE). Pass y to make the
    call itself allocate nothing (with y=None this wrapper allocates the output)."""
    M, K = x.shape
    N = _check_proj(packed, s_w, per_row, K)
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check_out(y, M, N)
    od = OUT_BF16 if y.dtype == torch.bfloat16 else OUT_F32
    _check(lib.bitnet_linear_noalloc(_x_ptr(x), M, K, _dev(packed, torch.uint8, "packed"),
                                     _dev(s_w, torch.float32, "s_w"), int(bool(per_row)), N,
                                     _dev(y, y.dtype, "y"), od, _stream(stream)),
           "bitnet_linear_noalloc")
    return y


def bitnet_pack_ternary_b3(t: torch.Tensor, stream=None) -> torch.Tensor:
    """Ternary (N, K) int8 -> the base-3 format, five weights per byte (N, 16 ceil(K / 80))."""
    N, K = t.shape
    packed = torch.empty((N, int(lib.bitnet_b3_row_bytes(K))), dtype=torch.uint8, device=t.device)
    _check(lib.bitnet_pack_ternary_b3(_dev(t, torch.int8, "t"), N, K, packed.data_ptr(),
                                      _stream(stream)), "bitnet_pack_ternary_b3")
    return packed


def bitnet_linear_b3(x: torch.Tensor, packed_b3: torch.Tensor, s_w: torch.Tensor, per_row: bool,
                     out_dtype: torch.dtype = torch.bfloat16, y: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """bitnet_linear for one token on base-3 weights (bitnet_pack_ternary_b3)."""
    M, K = x.shape
    N = packed_b3.shape[0]
    if packed_b3.dim() != 2 or packed_b3.shape[1] != int(lib.bitnet_b3_row_bytes(K)):
        raise ValueError("packed_b3 must be (N, bitnet_b3_row_bytes(K))")
    if s_w.numel() != (N if per_row else 1):
        raise ValueError("s_w must have N (per row) or 1 elements")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check_out(y, M, N)
    od = OUT_BF16 if y.dtype == torch.bfloat16 else OUT_F32
    _check(lib.bitnet_linear_b3(_x_ptr(x), M, K, _dev(packed_b3, torch.uint8, "packed_b3"),
                                _dev(s_w, torch.float32, "s_w"), int(bool(per_row)), N,
                                _dev(y, y.dtype, "y"), od, _stream(stream)), "bitnet_linear_b3")
    return y


# ----------------------------------------------------------------------------- decode step
# The operators of a decode step beside the ternary projections. They run on the device of their
# tensors, whichever is current. With `stream` given, what a call allocates belongs to that stream (no
# pending work of the current one can still be using it), and no tensor of a call, the cache's own
# among them, is reused before both streams are done with it. A call's host time is that of a decode
# step's, so the checks are few and flat.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
    lambda i: torch.cuda.current_stream(i).cuda_stream)
_current = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else (
    torch.cuda.current_device)


def _elsewhere(dev: int, call, *args, **kw):
    """call(...) with device `dev`, which is not the current one, made current."""
    if dev < 0:
        raise ValueError(f"{call.__name__}: the tensors must be on a CUDA device")
    with torch.cuda.device(dev):
        return call(*args, **kw)


def _handle(stream: Optional[torch.cuda.Stream], dev: int) -> int:
    if stream is None:
        return _raw_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _new(shape, dtype: torch.dtype, dev: torch.device, stream) -> torch.Tensor:
    """A tensor for a call on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(here)
    return t


def _keep(stream: torch.cuda.Stream, *tensors):
    """The caller's tensors are not to be reused before `stream` is done with them."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _on(t: torch.Tensor, dtype: torch.dtype, dev: int, name: str) -> int:
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}, got {t.dtype} "
                         f"on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))
    return t.data_ptr()


def bitnet_pack_w4(W: torch.Tensor, group: int = 128, stream=None):
    """Latent weights (N, K) fp32 -> 4-bit weights (N, 64 ceil(K / 128)) uint8 and their scales
    (N, ceil(K / group)) bf16, group = 32, 64 or 128."""
    dev = W.get_device()
    if W.dim() != 2:
        raise ValueError(f"W must be (N, K), got {tuple(W.shape)}")
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    if dev < 0 or dev != _current():
        return _elsewhere(dev, bitnet_pack_w4, W, group, stream)
    N, K = W.shape
    handle = _handle(stream, dev)
    packed = _new((N, -(-K // 128) * 64), torch.uint8, W.device, stream)
    scales = _new((N, -(-K // group)), torch.bfloat16, W.device, stream)
    _check(lib.bitnet_pack_w4(_on(W, torch.float32, dev, "W"), N, K, group, packed.data_ptr(),
                              scales.data_ptr(), handle), "bitnet_pack_w4")
    if stream is not None:
        _keep(stream, W)
    return packed, scales


def bitnet_linear_w4(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group: int,
                     out_dtype: torch.dtype = torch.bfloat16, y: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """y (M, N) = x (M, K) bf16 times 4-bit weights with group scales (bitnet_pack_w4). Behind a kernel
    other than bitnet_pack_w4 that changes weights or scales (not a copy), another torch kernel has to
    come first: the call reads them before its predecessor has ended."""
    M, K = x.shape
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    N, row_bytes = packed.shape
    if row_bytes != -(-K // 128) * 64 or scales.shape != (N, -(-K // group)):
        raise ValueError(f"packed must be (N, {-(-K // 128) * 64}) and scales (N, {-(-K // group)})"
                         f", got {tuple(packed.shape)} and {tuple(scales.shape)}")
    dev = x.get_device()
    if dev < 0 or dev != _current():
        return _elsewhere(dev, bitnet_linear_w4, x, packed, scales, group, out_dtype, y, stream)
    handle = _handle(stream, dev)
    if y is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        y = _new((M, N), out_dtype, x.device, stream)
        yp = y.data_ptr()
    else:
        _check_out(y, M, N)
        yp = _on(y, y.dtype, dev, "y")
    st = lib.bitnet_linear_w4(_on(x, torch.bfloat16, dev, "x"), M, K,
                              _on(packed, torch.uint8, dev, "packed"),
                              _on(scales, torch.bfloat16, dev, "scales"), group, N, yp,
                              OUT_BF16 if y.dtype is torch.bfloat16 else OUT_F32, handle)
    if st:
        _check(st, "bitnet_linear_w4")
    if stream is not None:
        _keep(stream, x, packed, scales, y)
    return y


class PagedCache:
    """A paged key/value cache over the caller's tensors (see bitnet.h for the layout).

    table  (max_seqs, max_pages) int32, lens (max_seqs) int32, refs (num_pages) int32.
    layers one (k, v) or (k, v, k_scale, v_scale) per layer: pools (num_pages, kv_heads,
           page_size, head_dim), bf16, or int8 with scales (num_pages, kv_heads, page_size) fp32.
    error  one int32 word of CACHE_ERR_* bits (allocated and cleared here if not given);
           errors() reads and clears it.
    make_cache allocates a new, empty one.
    """

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                 layers: Sequence, error: Optional[torch.Tensor] = None):
        dev = table.get_device()
        if dev < 0:
            raise ValueError(f"table must be a CUDA tensor, got {table.device}")
        if table.dim() != 2 or lens.shape != table.shape[:1] or refs.dim() != 1:
            raise ValueError("table must be (max_seqs, max_pages), lens (max_seqs), refs "
                             "(num_pages)")
        if not 1 <= len(layers) <= CACHE_MAX_LAYERS:
            raise ValueError(f"1..{CACHE_MAX_LAYERS} layers")
        k0 = layers[0][0]
        if k0.dim() != 4 or k0.shape[0] != refs.shape[0]:
            raise ValueError(f"pools must be ({refs.shape[0]}, kv_heads, page_size, head_dim), got "
                             f"{tuple(k0.shape)}")
        if k0.dtype not in (torch.bfloat16, torch.int8):
            raise ValueError(f"pools must be bfloat16 or int8, got {k0.dtype}")
        i8 = k0.dtype == torch.int8
        self.table, self.lens, self.refs = table, lens, refs
        self.layers = [tuple(layer) for layer in layers]
        self.device, self.dtype = table.device, k0.dtype
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k0.shape
        self.max_seqs, self.max_pages = table.shape
        if error is None:
            error = torch.zeros(1, dtype=torch.int32, device=table.device)
        if error.numel() != 1:
            raise ValueError("error must have 1 element")
        self.error = error
        self._dev = dev
        self._layers = (bitnet_cache_layer * len(layers))()
        for c_layer, layer in zip(self._layers, self.layers):
            pools, scales = layer[:2], [t for t in layer[2:] if t is not None]
            if len(pools) != 2 or len(scales) != (2 if i8 else 0):
                raise ValueError("a layer is (k, v) in bfloat16, or (k, v, k_scale, v_scale) in "
                                 "int8")
            if any(t.shape != k0.shape for t in pools) or \
                    any(t.shape != k0.shape[:3] for t in scales):
                raise ValueError("all pools must have one shape, scales (num_pages, kv_heads, "
                                 "page_size)")
            c_layer.k, c_layer.v = (_on(t, k0.dtype, dev, "pool") for t in pools)
            if i8:
                c_layer.k_scale, c_layer.v_scale = (_on(t, torch.float32, dev, "scale")
                                                    for t in scales)
        self._layer_refs = [ctypes.byref(c_layer) for c_layer in self._layers]
        self._tensors = [table, lens, refs, error] + [t for layer in self.layers for t in layer
                                                      if t is not None]
        self._streams = set()  # those that calls were given: see _keep
        self._c = bitnet_cache(_on(table, torch.int32, dev, "table"),
                               _on(lens, torch.int32, dev, "lens"),
                               _on(refs, torch.int32, dev, "refs"),
                               _on(error, torch.int32, dev, "error"), self.num_pages,
                               self.max_seqs, self.max_pages, self.page_size, self.kv_heads,
                               self.head_dim, CACHE_I8 if i8 else CACHE_BF16)
        self._ref = ctypes.byref(self._c)
        self._sizes = {}  # workspace bytes by call
        self._kept = threading.local()  # .ws: the default stream's workspace (see _scratch)

    def _layer(self, i: int):
        if not 0 <= i < len(self.layers):
            raise IndexError(f"layer {i} of {len(self.layers)}")
        return self._layer_refs[i]

    def _keep(self, stream: torch.cuda.Stream, *tensors):
        """Neither the cache's tensors nor these are to be reused before `stream` is done with them.
        The cache's are told once per stream: what the allocator notes of a tensor holds until it is
        freed, and covers what the stream was given until then."""
        if stream.cuda_stream not in self._streams:
            _keep(stream, *self._tensors)
            self._streams.add(stream.cuda_stream)
        _keep(stream, *tensors)

    def workspace_size(self, n: int) -> int:
        """Bytes of scratch for upkeep calls on lists of n slots."""
        size = self._sizes.get(n)
        if size is None:
            size = self._sizes[n] = int(lib.bitnet_cache_workspace_size(self._ref, n))
        return size

    def attention_workspace_size(self, B: int, heads: int) -> int:
        """Bytes of scratch for bitnet_paged_attention of B queries."""
        size = self._sizes.get((B, heads))
        if size is None:
            size = self._sizes[B, heads] = int(
                lib.bitnet_paged_attention_workspace_size(self._ref, B, heads))
        return size

    def errors(self) -> int:
        """Reads and clears the error word, once the device has done all that it was given before, on
        whichever stream. No other thread may make calls on the cache meanwhile: a bit that one sets
        between the reading and the clearing would be lost."""
        torch.cuda.synchronize(self.device)
        e = int(self.error.item())
        if e:
            self.error.zero_()
            torch.cuda.current_stream(self.device).synchronize()  # cleared before other streams go on
        return e


def make_cache(num_pages: int, max_seqs: int, max_pages: int, kv_heads: int, head_dim: int,
               page_size: int = 64, layers: int = 1, dtype: torch.dtype = torch.bfloat16,
               device=None) -> PagedCache:
    """A new, empty cache."""
    dev = torch.device(device or "cuda")
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    shape = (num_pages, kv_heads, page_size, head_dim)
    made = []
    for _ in range(layers):
        pools = [torch.zeros(shape, dtype=dtype, device=dev) for _ in range(2)]
        if dtype == torch.int8:
            pools += [torch.ones(shape[:3], dtype=torch.float32, device=dev) for _ in range(2)]
        made.append(tuple(pools))
    return PagedCache(torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                      torch.zeros(max_seqs, dtype=torch.int32, device=dev),
                      torch.zeros(num_pages, dtype=torch.int32, device=dev), made)


def _slots(cache: PagedCache, t: torch.Tensor, name: str, n: int) -> int:
    if t.shape != (n,):
        raise ValueError(f"{name} must be a list of {n}, got {tuple(t.shape)}")
    return _on(t, torch.int32, cache._dev, name)


def _scratch(cache: PagedCache, workspace: Optional[torch.Tensor], size: int, stream, handle: int):
    """The workspace of a call, its address and its bytes. A thread's calls on the legacy default
    stream share one that the cache keeps: they run one after the other (those of two threads may
    mix their kernels), and that stream cannot be captured, so no graph holds it. Other streams get
    a new one each time."""
    if workspace is None:
        if handle == 0 and stream is None:
            workspace = getattr(cache._kept, "ws", None)
            if workspace is None or workspace.shape[0] < size:
                workspace = cache._kept.ws = _new(size, torch.uint8, cache.device, None)
        else:
            workspace = _new(size, torch.uint8, cache.device, stream)
        return workspace, workspace.data_ptr(), size
    if workspace.get_device() != cache._dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {cache.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _copies(cache: PagedCache, room: int, copies: Optional[torch.Tensor], stream):
    """A list of page copies with room for `room` pairs: int32 [count, 0, from, to, from, ...]."""
    if copies is None:
        copies = _new(2 + 2 * room, torch.int32, cache.device, stream)
        return copies, copies.data_ptr(), room
    if copies.dim() != 1 or copies.shape[0] < 2 + 2 * room:
        raise ValueError(f"copies must be one list of at least {2 + 2 * room}")
    return copies, _on(copies, torch.int32, cache._dev, "copies"), (copies.shape[0] - 2) // 2


def bitnet_cache_fork(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Slots dst[i] (empty ones) become copies of slots src[i] that share their pages."""
    dev, n = cache._dev, src.shape[0]
    if dev != _current():
        return _elsewhere(dev, bitnet_cache_fork, cache, src, dst, workspace, stream)
    handle = _handle(stream, dev)
    ws, wp, wb = _scratch(cache, workspace, cache.workspace_size(n), stream, handle)
    st = lib.bitnet_cache_fork(cache._ref, _slots(cache, src, "src", n),
                               _slots(cache, dst, "dst", n), n, wp, wb, handle)
    if st:
        _check(st, "bitnet_cache_fork")
    if stream is not None:
        cache._keep(stream, src, dst, ws)


def bitnet_cache_extend(cache: PagedCache, seqs: torch.Tensor, add: torch.Tensor,
                        copies: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Slots seqs[i] grow by add[i] tokens. Returns the page copies that bitnet_cache_copy has
    to make before the tokens are written: int32 [count, 0, from, to, from, to, ...]."""
    dev, n = cache._dev, seqs.shape[0]
    if dev != _current():
        return _elsewhere(dev, bitnet_cache_extend, cache, seqs, add, copies, workspace, stream)
    handle = _handle(stream, dev)
    copies, cp, room = _copies(cache, n, copies, stream)
    ws, wp, wb = _scratch(cache, workspace, cache.workspace_size(n), stream, handle)
    st = lib.bitnet_cache_extend(cache._ref, _slots(cache, seqs, "seqs", n),
                                 _slots(cache, add, "add", n), n, cp, room, wp, wb, handle)
    if st:
        _check(st, "bitnet_cache_extend")
    if stream is not None:
        cache._keep(stream, seqs, add, copies, ws)
    return copies


def bitnet_cache_free(cache: PagedCache, seqs: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Slots seqs[i] become empty."""
    dev, n = cache._dev, seqs.shape[0]
    if dev != _current():
        return _elsewhere(dev, bitnet_cache_free, cache, seqs, workspace, stream)
    handle = _handle(stream, dev)
    ws, wp, wb = _scratch(cache, workspace, cache.workspace_size(n), stream, handle)
    st = lib.bitnet_cache_free(cache._ref, _slots(cache, seqs, "seqs", n), n, wp, wb, handle)
    if st:
        _check(st, "bitnet_cache_free")
    if stream is not None:
        cache._keep(stream, seqs, ws)


def bitnet_cache_compact(cache: PagedCache, copies: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the pages in use to the front of the pool. Returns the moves for bitnet_cache_copy,
    which must run before the cache is read or written again."""
    dev = cache._dev
    if dev != _current():
        return _elsewhere(dev, bitnet_cache_compact, cache, copies, workspace, stream)
    handle = _handle(stream, dev)
    copies, cp, room = _copies(cache, cache.num_pages // 2, copies, stream)
    ws, wp, wb = _scratch(cache, workspace, cache.workspace_size(0), stream, handle)
    st = lib.bitnet_cache_compact(cache._ref, cp, room, wp, wb, handle)
    if st:
        _check(st, "bitnet_cache_compact")
    if stream is not None:
        cache._keep(stream, copies, ws)
    return copies


def bitnet_cache_copy(cache: PagedCache, copies: torch.Tensor, stream=None) -> None:
    """Copies pages from -> to in every layer of the cache, for a list that bitnet_cache_extend or
    bitnet_cache_compact returned."""
    dev = cache._dev
    if dev != _current():
        return _elsewhere(dev, bitnet_cache_copy, cache, copies, stream)
    if copies.dim() != 1 or copies.shape[0] < 2:
        raise ValueError("copies must be [count, 0, from, to, ...]")
    st = lib.bitnet_cache_copy(cache._ref, cache._layers, len(cache.layers),
                               _on(copies, torch.int32, dev, "copies"),
                               (copies.shape[0] - 2) // 2, _handle(stream, dev))
    if st:
        _check(st, "bitnet_cache_copy")
    if stream is not None:
        cache._keep(stream, copies)


def bitnet_cache_append(cache: PagedCache, layer: int, k: torch.Tensor, v: torch.Tensor,
                        seqs: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """Writes T tokens, k and v (T, kv_heads, head_dim) or (T, kv_heads * head_dim) bf16, into a
    layer's pages: token t at position pos[t] (default: the last) of slot seqs[t] (default: t)."""
    dev, T = cache._dev, k.shape[0]
    if dev != _current():
        return _elsewhere(dev, bitnet_cache_append, cache, layer, k, v, seqs, pos, stream)
    flat, heads = (T, cache.kv_heads * cache.head_dim), (T, cache.kv_heads, cache.head_dim)
    if k.shape not in (flat, heads) or v.shape not in (flat, heads):
        raise ValueError(f"k and v must be (T, {cache.kv_heads}, {cache.head_dim}), got "
                         f"{tuple(k.shape)} and {tuple(v.shape)}")
    if seqs is None and T > cache.max_seqs:
        raise ValueError(f"{T} tokens for {cache.max_seqs} slots: give seqs")
    st = lib.bitnet_cache_append(
        cache._ref, cache._layer(layer), _on(k, torch.bfloat16, dev, "k"),
        _on(v, torch.bfloat16, dev, "v"), T,
        None if seqs is None else _slots(cache, seqs, "seqs", T),
        None if pos is None else _slots(cache, pos, "pos", T), _handle(stream, dev))
    if st:
        _check(st, "bitnet_cache_append")
    if stream is not None:
        cache._keep(stream, k, v, seqs, pos)


def bitnet_paged_attention(q: torch.Tensor, cache: PagedCache, layer: int = 0,
                           seqs: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                           window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
                           return_lse: bool = False, lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of one new token per sequence: q (B, heads, head_dim) or (B, heads * head_dim)
    bf16 over slot seqs[b] (default: b) of the cache. scale defaults to head_dim ** -0.5; window
    and sinks hide all but the first `sinks` and the last `window` tokens. Returns out (shaped as
    q), or (out, lse) with lse (B, heads) fp32 if return_lse or a tensor for it is given."""
    dev, D = cache._dev, cache.head_dim
    if dev != _current():
        return _elsewhere(dev, bitnet_paged_attention, q, cache, layer, seqs, scale, window, sinks,
                          out, return_lse, lse, workspace, stream)
    shape = q.shape
    B = shape[0]
    if len(shape) == 3 and shape[2] == D:
        heads = shape[1]
    elif len(shape) == 2 and shape[1] % D == 0:
        heads = shape[1] // D
    else:
        raise ValueError(f"q must be (B, heads, {D}), got {tuple(shape)}")
    if seqs is None and B > cache.max_seqs:
        raise ValueError(f"{B} queries for {cache.max_seqs} slots: give seqs")
    handle = _handle(stream, dev)
    qp = _on(q, torch.bfloat16, dev, "q")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(shape, q.dtype, q.device, stream)
        op = out.data_ptr()
    elif out.shape == shape:
        op = _on(out, torch.bfloat16, dev, "out")
    else:
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    lp = None
    if lse is not None:
        if lse.shape != (B, heads):
            raise ValueError(f"lse must be ({B}, {heads}), got {tuple(lse.shape)}")
        lp = _on(lse, torch.float32, dev, "lse")
    elif return_lse:
        lse = _new((B, heads), torch.float32, cache.device, stream)
        lp = lse.data_ptr()
    ws, wp, wb = _scratch(cache, workspace, cache.attention_workspace_size(B, heads), stream, handle)
    st = lib.bitnet_paged_attention(
        cache._ref, cache._layer(layer), qp, B, heads,
        None if seqs is None else _slots(cache, seqs, "seqs", B),
        D ** -0.5 if scale is None else scale, window, sinks, op, lp, wp, wb, handle)
    if st:
        _check(st, "bitnet_paged_attention")
    if stream is not None:
        cache._keep(stream, q, seqs, out, lse, ws)
    return out if lse is None else (out, lse)


def bitnet_act_amax(x: torch.Tensor, stream=None) -> torch.Tensor:
    """Per-token max |x| (fp32, exact), the first tensor-parallel step of a K-split projection."""
    M, K = x.shape
    amax = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitnet_act_amax(_x_ptr(x), M, K, amax.data_ptr(), _stream(stream)),
           "bitnet_act_amax")
    return amax


def bitnet_quant_act_amax(x: torch.Tensor, amax: torch.Tensor, stream=None):
    """Per-token quantiser with the amax supplied (e.g. all-reduced over a K split): (q, s_x)."""
    M, K = x.shape
    if amax.numel() != M:
        raise ValueError(f"amax must have {M} elements, got {amax.numel()}")
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s_x = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitnet_quant_act_amax(_x_ptr(x), M, K, _dev(amax, torch.float32, "amax"),
                                     q.data_ptr(), s_x.data_ptr(), _stream(stream)),
           "bitnet_quant_act_amax")
    return q, s_x


def bitnet_dequant(acc: torch.Tensor, s_x: torch.Tensor, s_w: torch.Tensor, per_row: bool,
                   out_dtype: torch.dtype = torch.bfloat16, y: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The epilogue alone on an int32 accumulator (M, N): y = acc * (s_w * (1 / s_x))."""
    M, N = acc.shape
    if s_x.numel() != M or s_w.numel() != (N if per_row else 1):
        raise ValueError("s_x must have M elements and s_w N (per row) or 1")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=acc.device)
    _check_out(y, M, N)
    od = OUT_BF16 if y.dtype == torch.bfloat16 else OUT_F32
    _check(lib.bitnet_dequant(_dev(acc, torch.int32, "acc"), M, N, _dev(s_x, torch.float32, "s_x"),
                              _dev(s_w, torch.float32, "s_w"), int(bool(per_row)),
                              _dev(y, y.dtype, "y"), od, _stream(stream)), "bitnet_dequant")
    return y


def bitnet_linear_plan(M: int, K: int, Ns: Sequence[int], swiglu: bool = False,
                       workspace_bytes: Optional[int] = None, path: int = PATH_AUTO) -> dict:
    """The kernels a bitnet_linear_batch (or, with swiglu, bitnet_linear_swiglu with
    Ns = [2I]) call would run: host-only, nothing is launched. workspace_bytes defaults to
    workspace_size(M, K), what make_workspace provides."""
    n = len(Ns)
    arr = (_I64 * max(n, 1))(*Ns)
    wb = workspace_size(M, K) if workspace_bytes is None else int(workspace_bytes)
    pl = bitnet_plan()
    _check(lib.bitnet_linear_plan(M, K, arr, n, int(bool(swiglu)), wb, path, ctypes.byref(pl)),
           "bitnet_linear_plan")
    return {"kernel": pl.kernel, "grid": pl.grid, "tile_tokens": pl.tile_tokens,
            "splits": pl.splits, "tile_rows": pl.tile_rows}


def bitnet_check_device_errors() -> int:
    flags = _I32(0)
    st = lib.bitnet_check_device_errors(ctypes.byref(flags))
    if st not in (OK, ERR_TIMEOUT):
        raise BitnetError(st, "bitnet_check_device_errors")
    return int(flags.value)


def bitnet_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launches the watchdog self-test: one bounded wait on a barrier nothing completes."""
    st = lib.bitnet_selftest_wait_timeout(int(limit_ns), _stream(stream))
    if st != OK:
        raise BitnetError(st, "bitnet_selftest_wait_timeout")


def bitnet_version() -> int:
    return int(lib.bitnet_version())
