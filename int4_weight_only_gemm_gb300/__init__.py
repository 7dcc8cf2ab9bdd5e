"""Python binding of the W4A16 group-quantized GEMM library (libw4a16.so).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/w4a16.h.  PyTorch supplies device
memory and streams.  There is no fallback: if the compiled library is missing
or a call fails, an exception is raised.

    y[m][n] = sum_k x[m][k] * (q[k][n] - z[k/128][n]) * s[k/128][n]

Tensors (all on one CUDA device, contiguous):
    x        [M, K]    torch.bfloat16
    qweight  [K/8, N]  torch.int32   canonical packing (bits 4i..4i+3 = row 8j+i)
    qweight_dev        torch.int32   device layout from w4a16_pack (same size)
    scales   [K/128, N] torch.float16
    qzeros   [K/128, N/8] torch.int32 (bits 4i..4i+3 = column 8c+i)
    y        [M, N]    torch.bfloat16
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a16.so")

W4A16_OK = 0
W4A16_EINVAL = -1
W4A16_EALIGN = -2
W4A16_EUNSUPPORTED = -3
W4A16_ECUDA = -4
W4A16_ETIMEOUT = -5
W4A16_EWORKSPACE = -6
PATH_AUTO, PATH_GEMV, PATH_TC, PATH_GEMV_SPLITK, PATH_GEMV_CS = 0, 1, 2, 3, 4
FLAG_PDL, FLAG_STATIC_WEIGHTS = 1, 2

_lib = None
_lock = threading.Lock()


class W4A16Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {w4a16_status_str(status)} (status {status})")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads the compiled library; raises if it has not been built."""
    global _lib
    if _lib is not None:  # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing: build it with "
                                  "`python -m int4_weight_only_gemm_gb300._build`")
            lib = ctypes.CDLL(path)
            vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
            lib.w4a16_pack.argtypes = [vp, vp, ci, ci, vp]
            lib.w4a16_requant_pack.argtypes = [vp, vp, vp, ci, ci, ci, vp, vp]
            lib.w4a16_unpack.argtypes = [vp, vp, ci, ci, vp]
            lib.w4a16_pack_gate_up.argtypes = [vp, vp, ci, ci, vp]
            lib.w4a16_unpack_gate_up.argtypes = [vp, vp, ci, ci, vp]
            lib.w4a16_gemm_gate_up_silu.argtypes = [ci, ctypes.c_uint, vp, vp, vp, vp, ci, ci, ci, ci, vp, vp, sz, vp]
            lib.w4a16_workspace_bytes.argtypes = [ci, ci, ci, ci]
            lib.w4a16_workspace_bytes.restype = sz
            lib.w4a16_workspace_bytes_max.argtypes = [ci, ci, ci, ci]
            lib.w4a16_workspace_bytes_max.restype = sz
            lib.w4a16_workspace_bytes_path.argtypes = [ci, ci, ci, ci, ci]
            lib.w4a16_workspace_bytes_path.restype = sz
            lib.w4a16_set_workspace.argtypes = [vp, sz]
            lib.w4a16_gemm.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, vp, vp]
            lib.w4a16_gemm_ws.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, vp, vp, sz, vp]
            lib.w4a16_gemm_path.argtypes = [ci, vp, vp, vp, vp, ci, ci, ci, ci, vp, vp, sz, vp]
            lib.w4a16_gemm_ex.argtypes = [ci, ctypes.c_uint, vp, vp, vp, vp, ci, ci, ci, ci, vp, vp, sz, vp]
            lib.w4a16_auto_path.argtypes = [ci, ci, ci, ci]
            lib.w4a16_status_str.argtypes = [ci]
            lib.w4a16_status_str.restype = ctypes.c_char_p
            lib.w4a16_last_device_status.argtypes = [vp]
            lib.w4a16_launch_count.restype = ctypes.c_uint64
            lib.w4a16_swa_attention.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, ci, vp, vp, sz,
                                                ctypes.c_uint, vp]
            lib.w4a16_swa_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci, ci]
            lib.w4a16_swa_workspace_bytes.restype = sz
            for name in ("w4a16_page_plan", "w4a16_kv_write", "w4a16_paged_attention", "w4a16_sample"):
                getattr(lib, name).argtypes = [ctypes.c_char_p, vp]  # a packed argument struct, a stream
            lib.w4a16_paged_attention_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci]
            lib.w4a16_paged_attention_workspace_bytes.restype = sz
            lib.w4a16_sample_workspace_bytes.argtypes = [ci, ci, ci]
            lib.w4a16_sample_workspace_bytes.restype = sz
            lib.w4a16_stream_capture_id.argtypes = [vp]
            lib.w4a16_stream_capture_id.restype = ctypes.c_uint64
            _lib = lib
    return _lib


# the current stream's handle without building a Stream object (a few
# microseconds a call); the public route where this torch lacks it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device_index: int | None = None) -> int:
    if stream is None:
        if _raw_stream is not None:
            return int(_raw_stream(torch.cuda.current_device() if device_index is None else device_index))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _raise(status: int, what: str):
    if status != W4A16_OK:
        raise W4A16Error(status, what)


def w4a16_status_str(status: int) -> str:
    return load_library().w4a16_status_str(int(status)).decode()


def w4a16_pack(qweight: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Canonical [K/8, N] int32 codes -> device layout (same size)."""
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    _check(qweight, "qweight", torch.int32)
    if out is None:
        out = torch.empty_like(qweight)
    _check(out, "out", torch.int32, qweight.shape)
    _raise(load_library().w4a16_pack(qweight.data_ptr(), out.data_ptr(), K, N, _stream(stream)), "w4a16_pack")
    return out


def w4a16_requant_pack(w: torch.Tensor, scales: torch.Tensor, qzeros: torch.Tensor, group: int = 128,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Re-quantize bf16 w [K, N] onto the frozen grid (scales, qzeros) straight
    into the device layout: code = clamp(round(w / s) + z, 0, 15)."""
    _check(w, "w", torch.bfloat16)
    if w.dim() != 2:
        raise ValueError("w must be [K, N]")
    K, N = w.shape
    G = K // group
    _check(scales, "scales", torch.float16, (G, N))
    _check(qzeros, "qzeros", torch.int32, (G, N // 8))
    if out is None:
        out = torch.empty((K // 8, N), dtype=torch.int32, device=w.device)
    _check(out, "out", torch.int32, (K // 8, N))
    _raise(load_library().w4a16_requant_pack(w.data_ptr(), scales.data_ptr(), qzeros.data_ptr(), K, N, group,
                                             out.data_ptr(), _stream(stream)), "w4a16_requant_pack")
    return out


def w4a16_unpack(qweight_dev: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Device layout -> canonical [K/8, N] int32 (exact inverse of w4a16_pack)."""
    _check(qweight_dev, "qweight_dev", torch.int32)
    K, N = qweight_dev.shape[0] * 8, qweight_dev.shape[1]
    if out is None:
        out = torch.empty_like(qweight_dev)
    _check(out, "out", torch.int32, qweight_dev.shape)
    _raise(load_library().w4a16_unpack(qweight_dev.data_ptr(), out.data_ptr(), K, N, _stream(stream)),
           "w4a16_unpack")
    return out


def w4a16_pack_gate_up(qweight: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Canonical [K/8, 2H] int32 codes of fused gate/up weights (gate columns
    first) -> the interleaved device layout of w4a16_gemm_gate_up_silu."""
    _check(qweight, "qweight", torch.int32)
    K, H = qweight.shape[0] * 8, qweight.shape[1] // 2
    if out is None:
        out = torch.empty_like(qweight)
    _check(out, "out", torch.int32, qweight.shape)
    _raise(load_library().w4a16_pack_gate_up(qweight.data_ptr(), out.data_ptr(), K, H, _stream(stream)),
           "w4a16_pack_gate_up")
    return out


def w4a16_unpack_gate_up(qweight_dev: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Exact inverse of w4a16_pack_gate_up."""
    _check(qweight_dev, "qweight_dev", torch.int32)
    K, H = qweight_dev.shape[0] * 8, qweight_dev.shape[1] // 2
    if out is None:
        out = torch.empty_like(qweight_dev)
    _check(out, "out", torch.int32, qweight_dev.shape)
    _raise(load_library().w4a16_unpack_gate_up(qweight_dev.data_ptr(), out.data_ptr(), K, H, _stream(stream)),
           "w4a16_unpack_gate_up")
    return out


def w4a16_gemm_gate_up_silu(x: torch.Tensor, qweight_dev: torch.Tensor, scales: torch.Tensor,
                            qzeros: torch.Tensor, group: int = 128, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, path: int = PATH_AUTO, stream=None,
                            flags: int | None = None) -> torch.Tensor:
    """y = silu(x . Wg) * (x . Wu) in bf16 [M, H] for fused gate/up weights
    [K, 2H] packed by w4a16_pack_gate_up (scales / qzeros canonical, [G, 2H]
    and [G, 2H/8])."""
    _check(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    N = qweight_dev.shape[1]
    H = N // 2
    G = K // group if group > 0 else 0
    _check(qweight_dev, "qweight_dev", torch.int32, (K // 8, N))
    _check(scales, "scales", torch.float16, (G, N))
    _check(qzeros, "qzeros", torch.int32, (G, N // 8))
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", torch.bfloat16, (M, H))
    lib = load_library()
    if workspace is None:
        need = _workspace_need(path, M, N, K, group, x.device)
        if need:
            workspace = _cached_workspace(need, x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.w4a16_gemm_gate_up_silu(path, FLAG_PDL if flags is None else flags, x.data_ptr(),
                                     qweight_dev.data_ptr(), scales.data_ptr(), qzeros.data_ptr(), M, H, K, group,
                                     out.data_ptr(), ws_ptr, ws_bytes, _stream(stream))
    _raise(st, "w4a16_gemm_gate_up_silu")
    return out


def w4a16_workspace_bytes(M: int, N: int, K: int, group: int = 128, path: int = PATH_AUTO) -> int:
    return int(load_library().w4a16_workspace_bytes_path(path, M, N, K, group))


def w4a16_workspace_bytes_max(max_M: int, N: int, K: int, group: int = 128) -> int:
    return int(load_library().w4a16_workspace_bytes_max(max_M, N, K, group))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled workspace buffer (the library needs it zeroed once)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def w4a16_set_workspace(workspace: torch.Tensor | None) -> None:
    lib = load_library()
    if workspace is None:
        _raise(lib.w4a16_set_workspace(None, 0), "w4a16_set_workspace")
    else:
        _raise(lib.w4a16_set_workspace(workspace.data_ptr(), workspace.numel() * workspace.element_size()),
               "w4a16_set_workspace")


_ws_cache: dict[int, torch.Tensor] = {}
_need_cache: dict[tuple, int] = {}


def _remember(key: tuple, need: int) -> int:
    """Keeps a workspace's size; all of them go where sizes keep changing."""
    if len(_need_cache) >= 4096:
        _need_cache.clear()
    _need_cache[key] = int(need)
    return int(need)


def _workspace_need(path: int, M: int, N: int, K: int, group: int, device: torch.device) -> int:
    """Workspace bytes a problem needs, asked of the library once per problem
    and device (the answer depends only on these)."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    key = (path, M, N, K, group, idx)
    need = _need_cache.get(key)
    if need is None:
        need = _remember(key, load_library().w4a16_workspace_bytes_path(path, M, N, K, group))
    return need


def _cached_workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    idx = device.index if device.index is not None else torch.cuda.current_device()
    ws = _ws_cache.get(idx)
    if ws is None or ws.numel() < nbytes:
        ws = new_workspace(nbytes, device)
        _ws_cache[idx] = ws
    return ws


def w4a16_gemm(x: torch.Tensor, qweight_dev: torch.Tensor, scales: torch.Tensor, qzeros: torch.Tensor,
               group: int = 128, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               path: int = PATH_AUTO, stream=None, flags: int | None = None) -> torch.Tensor:
    """y = x . dequant(qweight_dev, scales, qzeros) in bf16, on the GPU kernels.

    flags=None uses the library's default launch flags; otherwise a mask of
    FLAG_PDL and FLAG_STATIC_WEIGHTS (see include/w4a16.h)."""
    _check(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    N = qweight_dev.shape[1]
    G = K // group if group > 0 else 0
    _check(qweight_dev, "qweight_dev", torch.int32, (K // 8, N))
    _check(scales, "scales", torch.float16, (G, N))
    _check(qzeros, "qzeros", torch.int32, (G, N // 8))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", torch.bfloat16, (M, N))
    lib = load_library()
    if workspace is None:
        need = _workspace_need(path, M, N, K, group, x.device)
        if need:
            workspace = _cached_workspace(need, x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    sp = _stream(stream, x.device.index)
    if flags is None:
        st = lib.w4a16_gemm_path(path, x.data_ptr(), qweight_dev.data_ptr(), scales.data_ptr(), qzeros.data_ptr(),
                                 M, N, K, group, out.data_ptr(), ws_ptr, ws_bytes, sp)
    else:
        st = lib.w4a16_gemm_ex(path, flags, x.data_ptr(), qweight_dev.data_ptr(), scales.data_ptr(),
                               qzeros.data_ptr(), M, N, K, group, out.data_ptr(), ws_ptr, ws_bytes, sp)
    _raise(st, "w4a16_gemm")
    return out


def w4a16_gemm_raw(x_ptr: int, qd_ptr: int, scales_ptr: int, qzeros_ptr: int, M: int, N: int, K: int,
                   group: int, y_ptr: int, ws_ptr: int | None, ws_bytes: int, path: int = PATH_AUTO,
                   stream: int = 0, flags: int | None = None) -> int:
    """Pointer-level call (no checks beyond the library's own), for timing loops."""
    lib = load_library()
    if flags is None:
        return lib.w4a16_gemm_path(path, x_ptr, qd_ptr, scales_ptr, qzeros_ptr, M, N, K, group, y_ptr,
                                   ws_ptr, ws_bytes, stream)
    return lib.w4a16_gemm_ex(path, flags, x_ptr, qd_ptr, scales_ptr, qzeros_ptr, M, N, K, group, y_ptr,
                             ws_ptr, ws_bytes, stream)


def w4a16_auto_path(M: int, N: int, K: int, group: int = 128) -> int:
    return int(load_library().w4a16_auto_path(M, N, K, group))


def w4a16_last_device_status(stream=None) -> int:
    status = int(load_library().w4a16_last_device_status(_stream(stream)))
    if status == W4A16_ETIMEOUT:  # a kernel that gave up may have left its workspace's counters above zero
        _stream_workspaces.clear()
    return status


def w4a16_launch_count() -> int:
    return int(load_library().w4a16_launch_count())


def w4a16_swa_workspace_bytes(nq: int, Hq: int, Hkv: int, L: int, window: int, block: bool = False,
                              head_dim: int = 128) -> int:
    return int(load_library().w4a16_swa_workspace_bytes(nq, Hq, Hkv, head_dim, L, window, int(block)))


def w4a16_swa_attention(q: torch.Tensor, k_cache: torch.Tensor, vt_cache: torch.Tensor, L: int, window: int,
                        block: bool = False, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None, flags: int = FLAG_PDL) -> torch.Tensor:
    """Sliding-window decode attention of a block of nq queries at positions
    L-nq .. L-1 (see include/w4a16.h).

    q [nq, Hq, 128] bf16; k_cache [Hkv, Lmax, 128] bf16; vt_cache [Hkv, 128,
    Lmax] bf16 (values transposed per head); returns out [nq, Hq, 128] bf16."""
    _check(q, "q", torch.bfloat16)
    _check(k_cache, "k_cache", torch.bfloat16)
    _check(vt_cache, "vt_cache", torch.bfloat16)
    if q.dim() != 3 or k_cache.dim() != 3 or vt_cache.dim() != 3:
        raise ValueError("q, k_cache, vt_cache must be 3-D")
    nq, Hq, d = q.shape
    Hkv, Lmax, _ = k_cache.shape
    if tuple(vt_cache.shape) != (Hkv, d, Lmax):
        raise ValueError(f"vt_cache has shape {tuple(vt_cache.shape)}, expected {(Hkv, d, Lmax)}")
    if out is None:
        out = torch.empty_like(q)
    _check(out, "out", torch.bfloat16, q.shape)
    lib = load_library()
    need = int(lib.w4a16_swa_workspace_bytes(nq, Hq, Hkv, d, L, window, int(block)))
    if workspace is None:
        workspace = _cached_workspace(max(need, 1), q.device)
    st = lib.w4a16_swa_attention(q.data_ptr(), k_cache.data_ptr(), vt_cache.data_ptr(), nq, Hq, Hkv, d, L, Lmax,
                                 window, int(block), out.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), flags, _stream(stream))
    _raise(st, "w4a16_swa_attention")
    return out


# ---------------------------------------------------------------------------
# serving: paged cache and sampling (see include/w4a16.h)
# ---------------------------------------------------------------------------
# The argument structs of the C ABI, packed by position (native sizes, no
# padding: the fields are ordered by size).
_PLAN_ARGS = struct.Struct("=9QqiiiiiI")
_WRITE_ARGS = struct.Struct("=5Q10qiiiiiiIi")
_ATTN_ARGS = struct.Struct("=9QQ11qiiiiiiiiiiiifI")
_SAMPLE_ARGS = struct.Struct("=9QQqqiiiI")
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_Tensor, _I32 = torch.Tensor, torch.int32  # (looked up some ten times a call)


def _int32(t, name, n=None):
    """Address of a contiguous int32 CUDA tensor, of that many entries."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype is not _I32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if n is not None and (t.numel() != n or t.dim() != 1):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n,)}")
    return t.data_ptr()


def _block_table(t, requests):
    """Columns and row stride of a block table."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype is not _I32 or t.dim() != 2:
        raise ValueError("block_table must be a 2-D int32 CUDA tensor")
    rows, columns = t.shape
    row, column = t.stride()
    if rows != requests or (column != 1 and columns > 1 and requests > 0):
        raise ValueError(f"block_table must be [{requests}, columns] with contiguous rows")
    return columns, row if requests > 1 else columns


def _strided(t, name, dtype, dims):
    """Shape and strides of a CUDA tensor of that many dimensions whose last one is contiguous."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(stride) != dims or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be {dims}-D with a contiguous last dimension")
    return shape, stride


# Workspaces of the calls that bring none: one a stream, so that calls on two
# streams never share counters or partial results.  A capture never takes an
# eager call's buffer, since its graph may be replayed beside that stream's
# calls: it has one of its own for each of its streams, out of the graph's
# memory, with the zeroing of its counters as a node of the graph.
_stream_workspaces: dict = {}   # (device, stream): buffer
_capture_workspaces: dict = {}  # (device, stream): (capture, buffer), kept for the capture's next call
_MOST_STREAMS = 64              # that keep a buffer; the one given longest ago goes first


def _stream_of(index: int, stream: int):
    """The stream of a raw handle.  0 and 1 are the default stream, which ExternalStream cannot name: it takes 0 for
    "none given" and hands out a stream of its pool, unordered with the default one."""
    return torch.cuda.default_stream(index) if stream in (0, 1) else torch.cuda.ExternalStream(stream, device=index)


def _zeroed(nbytes: int, index: int, stream: int) -> torch.Tensor:
    """A workspace made and its counters (all that has to be zero) zeroed on that stream."""
    with torch.cuda.stream(_stream_of(index, stream)):
        ws = torch.empty(max(nbytes, 65536), dtype=torch.uint8, device=f"cuda:{index}")
        ws[:65536].zero_()
    return ws


def _serving_workspace(nbytes: int, index: int, stream, handle: int) -> torch.Tensor:
    """The workspace of a call that brings none; `stream` as the caller gave it, `handle` what it stands for."""
    if stream is None:
        capturing = torch.cuda.is_current_stream_capturing()
    else:
        capturing = load_library().w4a16_stream_capture_id(handle) != 0
    if capturing:
        return _capture_workspace(nbytes, index, handle)
    if _capture_workspaces:
        _capture_workspaces.clear()  # (their captures are over, or take new ones)
    ws = _stream_workspaces.get((index, handle))
    if ws is not None and ws.numel() >= nbytes:
        return ws
    # Buffers that go are the stream's own: their memory is given out again in the order of that stream, behind the
    # kernels that still use it.
    fresh = _zeroed(max(nbytes, 2 * ws.numel() if ws is not None else 0), index, handle)
    if ws is None and len(_stream_workspaces) >= _MOST_STREAMS:
        del _stream_workspaces[next(iter(_stream_workspaces))]
    _stream_workspaces[(index, handle)] = fresh
    return fresh


def _capture_workspace(nbytes: int, index: int, handle: int) -> torch.Tensor:
    capture = load_library().w4a16_stream_capture_id(handle)
    held, ws = _capture_workspaces.get((index, handle), (0, None))
    if held != capture or ws.numel() < nbytes:
        ws = _zeroed(max(nbytes, 2 * ws.numel() if held == capture else 0), index, handle)
        _capture_workspaces[(index, handle)] = capture, ws
    return ws


def w4a16_page_plan(past_len: torch.Tensor, new_len: torch.Tensor, free_pages: torch.Tensor,
                    block_table: torch.Tensor, page_size: int, q_start: torch.Tensor | None = None,
                    kv_len: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                    slot_map: torch.Tensor | None = None, pages_used: torch.Tensor | None = None,
                    max_tokens: int | None = None, stream=None, flags: int = FLAG_PDL):
    """Block tables, slot map and positions of a step, on the GPU, from the
    requests' cached and new lengths (int32 [B]; see include/w4a16.h).

    block_table [B, columns] int32 is updated in place: the pages a request
    holds stay, the ones it needs now are taken from free_pages in request
    order, the rest becomes -1.  Returns (q_start [B+1], kv_len [B], positions
    [T], slot_map [T], pages_used [1]), all int32; T is slot_map's length, or
    max_tokens where slot_map is None (entries past the new tokens are -1)."""
    B = past_len.shape[0]
    past, new, free = _int32(past_len, "past_len", B), _int32(new_len, "new_len", B), _int32(free_pages, "free_pages")
    columns, row = _block_table(block_table, B)
    if slot_map is None:
        if max_tokens is None:
            raise ValueError("give slot_map or max_tokens")
        slot_map = torch.empty(max_tokens, dtype=torch.int32, device=past_len.device)
    T = slot_map.shape[0]
    if positions is None:
        positions = torch.empty(T, dtype=torch.int32, device=past_len.device)
    if q_start is None:
        q_start = torch.empty(B + 1, dtype=torch.int32, device=past_len.device)
    if kv_len is None:
        kv_len = torch.empty(B, dtype=torch.int32, device=past_len.device)
    if pages_used is None:
        pages_used = torch.empty(1, dtype=torch.int32, device=past_len.device)
    args = _PLAN_ARGS.pack(past, new, free, block_table.data_ptr(), _int32(q_start, "q_start", B + 1),
                           _int32(kv_len, "kv_len", B), _int32(positions, "positions", T),
                           _int32(slot_map, "slot_map", T), _int32(pages_used, "pages_used", 1), row, B,
                           free_pages.numel(), columns, T, page_size, flags)
    _raise(load_library().w4a16_page_plan(args, _stream(stream, past_len.get_device())), "w4a16_page_plan")
    return q_start, kv_len, positions, slot_map, pages_used


def _caches(k_cache, v_cache, dtype):
    """Shape of both caches, and their strides."""
    shape, ks = _strided(k_cache, "k_cache", dtype, 4)
    vshape, vs = _strided(v_cache, "v_cache", dtype, 4)
    if vshape != shape:
        raise ValueError(f"v_cache has shape {tuple(vshape)}, expected {tuple(shape)}")
    return shape, ks, vs


def w4a16_kv_write(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, stream=None, flags: int = FLAG_PDL) -> None:
    """New keys and values [T, heads, head_dim] (bf16 or fp16; strided views
    such as slices of a fused projection's output) into the caches [pages,
    heads, page_size, head_dim] at the slots of slot_map [T] (int32; negative
    or past the cache: skipped)."""
    dtype = k.dtype
    shape, (kt, kh, _) = _strided(k, "k", dtype, 3)
    vshape, (vt, vh, _) = _strided(v, "v", dtype, 3)
    if vshape != shape:
        raise ValueError(f"v has shape {tuple(vshape)}, expected {tuple(shape)}")
    T, heads, d = shape
    (pages, ch, page, cd), (kcp, kch, kcs, _), (vcp, vch, vcs, _) = _caches(k_cache, v_cache, dtype)
    if ch != heads or cd != d or dtype not in _DTYPES:
        raise ValueError(f"caches of {ch} heads of {cd} do not take k of {heads} heads of {d} in {dtype}")
    args = _WRITE_ARGS.pack(k.data_ptr(), v.data_ptr(), _int32(slot_map, "slot_map", T), k_cache.data_ptr(),
                            v_cache.data_ptr(), kt, kh, vt, vh, kcp, kch, kcs, vcp, vch, vcs, T, heads, d, pages, page,
                            _DTYPES[dtype], flags, 0)
    _raise(load_library().w4a16_kv_write(args, _stream(stream, k.get_device())), "w4a16_kv_write")


def w4a16_paged_attention_workspace_bytes(tokens: int, requests: int, q_heads: int, kv_heads: int, head_dim: int,
                                          max_q: int) -> int:
    return int(load_library().w4a16_paged_attention_workspace_bytes(tokens, requests, q_heads, kv_heads, head_dim,
                                                                    max_q))


def w4a16_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                          q_start: torch.Tensor, kv_len: torch.Tensor, max_q: int, window: int = 0,
                          block: bool = False, scale: float | None = None, out: torch.Tensor | None = None,
                          lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
                          flags: int = FLAG_PDL) -> torch.Tensor:
    """Attention of every request's new tokens over its paged cache (see
    include/w4a16.h): decode, draft blocks, prompt chunks and mixtures of them.

    q [T, Hq, d] bf16 or fp16, d 64 or 128; caches [pages, Hkv, page_size, d];
    block_table [B, columns], q_start [B+1], kv_len [B] int32; max_q at least
    every request's number of new tokens.  window = 0: no window.  lse: [T, Hq]
    f32, filled if given.  Returns out [T, Hq, d]."""
    dtype = q.dtype
    shape, (qt, qh, _) = _strided(q, "q", dtype, 3)
    T, Hq, d = shape
    (pages, Hkv, page, cd), (kcp, kch, kcs, _), (vcp, vch, vcs, _) = _caches(k_cache, v_cache, dtype)
    if cd != d or dtype not in _DTYPES:
        raise ValueError(f"caches with heads of {cd} do not go with q with heads of {d} in {dtype}")
    B = kv_len.shape[0]
    kv, start = _int32(kv_len, "kv_len", B), _int32(q_start, "q_start", B + 1)
    columns, row = _block_table(block_table, B)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=dtype, device=q.device)
    oshape, (ot, oh, _) = _strided(out, "out", dtype, 3)
    if oshape != shape:
        raise ValueError(f"out has shape {tuple(oshape)}, expected {tuple(shape)}")
    if lse is not None:
        _check(lse, "lse", torch.float32, (T, Hq))
    lib, idx = load_library(), q.get_device()
    st = _stream(stream, idx)
    if workspace is None:
        key = ("paged_attention", Hq, Hkv, d, max_q, idx)
        need = _need_cache.get(key)
        if need is None:  # for as many tokens and requests as a call takes, which change from step to step
            need = _remember(key, lib.w4a16_paged_attention_workspace_bytes(0x7fffffff // max(Hq, 1), 16384, Hq, Hkv,
                                                                            d, max_q))
        if need:
            workspace = _serving_workspace(need, idx, stream, st)
    elif not isinstance(workspace, _Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    args = _ATTN_ARGS.pack(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), start, kv,
                           out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                           0 if workspace is None else workspace.data_ptr(),
                           0 if workspace is None else workspace.numel() * workspace.element_size(), qt, qh, ot, oh,
                           kcp, kch, kcs, vcp, vch, vcs, row, T, B, Hq, Hkv, d, pages, page, columns, max_q, window,
                           int(block), _DTYPES[dtype], 0.0 if scale is None else scale, flags)
    _raise(lib.w4a16_paged_attention(args, st), "w4a16_paged_attention")
    return out


def _rows_of(t, name, dtype, rows):
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if t.numel() != rows or t.dim() != 1:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows,)}")
    return t.data_ptr()


def w4a16_sample_workspace_bytes(rows: int, vocab: int, filters: bool = True) -> int:
    return int(load_library().w4a16_sample_workspace_bytes(rows, vocab, int(filters)))


def w4a16_sample(logits: torch.Tensor, noise: torch.Tensor, temperature: torch.Tensor | None = None,
                 top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                 min_p: torch.Tensor | None = None, token: torch.Tensor | None = None,
                 logprob: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
                 flags: int = FLAG_PDL) -> torch.Tensor:
    """One token a row of logits [R, V] (bf16, fp16 or f32), filtered by each
    row's top-k, top-p and min-p at its temperature, drawn with the given
    exponential random numbers noise [R, V] f32 (see include/w4a16.h).

    temperature, top_p, min_p f32 [R] and top_k int32 [R], or None.  Returns
    token [R] int32; logprob [R] f32 is filled if given."""
    dtype = logits.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"logits must be bf16, fp16 or f32, got {dtype}")
    shape, (lr, _) = _strided(logits, "logits", dtype, 2)
    nshape, (nr, _) = _strided(noise, "noise", torch.float32, 2)
    if nshape != shape:
        raise ValueError(f"noise has shape {tuple(nshape)}, expected {tuple(shape)}")
    R, V = shape
    if token is None:
        token = torch.empty(R, dtype=torch.int32, device=logits.device)
    f32 = torch.float32
    lib, idx = load_library(), logits.get_device()
    st = _stream(stream, idx)
    if workspace is None:
        filters = top_k is not None or top_p is not None or min_p is not None
        key = ("sample", R, V, filters, idx)
        need = _need_cache.get(key)
        if need is None:
            need = _remember(key, lib.w4a16_sample_workspace_bytes(R, V, int(filters)))
        if need:
            workspace = _serving_workspace(need, idx, stream, st)
    elif not isinstance(workspace, _Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    args = _SAMPLE_ARGS.pack(logits.data_ptr(), noise.data_ptr(), _rows_of(temperature, "temperature", f32, R),
                             _rows_of(top_k, "top_k", torch.int32, R), _rows_of(top_p, "top_p", f32, R),
                             _rows_of(min_p, "min_p", f32, R), _rows_of(token, "token", torch.int32, R),
                             _rows_of(logprob, "logprob", f32, R),
                             0 if workspace is None else workspace.data_ptr(),
                             0 if workspace is None else workspace.numel() * workspace.element_size(),
                             lr if R > 1 else V, nr if R > 1 else V, R, V, _DTYPES[dtype], flags)
    _raise(lib.w4a16_sample(args, st), "w4a16_sample")
    return token


def to_device(problem, device="cuda"):
    """Host arrays of a w4a16_inputs.Problem -> CUDA tensors in the ABI dtypes."""
    import numpy as np
    x = torch.from_numpy(np.ascontiguousarray(problem.x).view(np.int16)).view(torch.bfloat16).to(device)
    qw = torch.from_numpy(np.ascontiguousarray(problem.qweight).view(np.int32)).to(device)
    sc = torch.from_numpy(np.ascontiguousarray(problem.scales).view(np.float16)).to(device)
    qz = torch.from_numpy(np.ascontiguousarray(problem.qzeros).view(np.int32)).to(device)
    return x, qw, sc, qz
