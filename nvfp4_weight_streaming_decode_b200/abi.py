"""ctypes binding of libnvfp4decode.so -- argument marshalling only.

Every function named ``nvfp4_*`` here has the C signature of the same name in
``include/nvfp4decode.h`` and returns its status (``NVFP4_OK`` = 0).  Device
pointers and streams are plain integers (``tensor.data_ptr()``,
``torch.cuda.current_stream().cuda_stream``).  The torch helpers at the end
only allocate device memory and pass pointers; all compute runs in the
library's CUDA kernels.  If the library is missing this module raises: there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
# NVFP4_LIB may name another build of the same library (same ABI).
LIB_PATH = os.environ.get("NVFP4_LIB") or os.path.join(HERE, "libnvfp4decode.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "nvfp4decode.h")

NVFP4_OK = 0
NVFP4_ERR_ARG = -1
NVFP4_ERR_M = -2
NVFP4_ERR_SHAPE = -3
NVFP4_ERR_ALIGN = -4
NVFP4_ERR_BAD_SCALE = -5
NVFP4_ERR_CUDA = -6
NVFP4_ERR_CAPTURE = -7
NVFP4_ERR_DEVICE = -8
NVFP4_ERR_SCRATCH = -9
NVFP4_ROUND_PERSISTENT = 0
NVFP4_ROUND_CHAIN = 1
NVFP4_DESC_GEMM = 0
NVFP4_DESC_GATEUP_SILU = 1
NVFP4_DESC_ROPE_APPEND = 2
NVFP4_DESC_ATTN_TREE = 3
NVFP4_TOPK_MAX_ROWS = 64
NVFP4_TOPK_MAX_K = 64
NVFP4_TOPK_MAX_V = 1 << 24
NVFP4_GROUPED_MAX_ROUTES = 128
NVFP4_CACHE_MAX_LANES = 64
NVFP4_ROPE_HALVES = 0
NVFP4_ROPE_ADJACENT = 1
NVFP4_ATTN_MAX_ROWS = 64
NVFP4_MAX_M = 64          # nvfp4_gemm_decode: 1..8 decode lanes, 9..64 verify rows
NVFP4_ROUND_ROWS = 8      # rows of a round's widest graph

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_I = ctypes.c_int
_I32 = ctypes.c_int32


class Nvfp4Cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("table", _P), ("len", _P), ("ref", _P), ("scratch", _P), ("layers", _I32),
                ("pages", _I32), ("kv_heads", _I32), ("page_size", _I32), ("head_dim", _I32), ("lanes", _I32),
                ("max_pages", _I32), ("reserved", _I32)]


class Nvfp4RopeArgs(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(Nvfp4Cache)), ("layer", _I32), ("rows", _I32), ("q_heads", _I32),
                ("rot_dim", _I32), ("style", _I32), ("axes", _I32), ("y", _P), ("ldy", _I64), ("row_start", _P),
                ("positions", _P), ("ldp", _I64), ("pair_axis", _P), ("inv_freq", _P), ("q", _P), ("ldq", _I64)]


class Nvfp4AttnArgs(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(Nvfp4Cache)), ("layer", _I32), ("rows", _I32), ("q_heads", _I32),
                ("max_nodes", _I32), ("scale", _F), ("reserved", _I32), ("q", _P), ("ldq", _I64), ("row_start", _P),
                ("mask", _P), ("out", _P), ("ldo", _I64), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_uint64)]


# The two argument structs as one native-layout record each: filling a ctypes
# structure field by field costs microseconds that a decode step would feel.
_ROPE_ARGS = struct.Struct("@P6iPqPPqPPPq")
_ATTN_ARGS = struct.Struct("@P4ifiPqPPPqPPQ")


class Nvfp4Expert(ctypes.Structure):
    _fields_ = [("wq", _P), ("ws", _P), ("gscale", _F), ("reserved", ctypes.c_int32)]


class Nvfp4GemmDesc(ctypes.Structure):
    _fields_ = [("kind", _I), ("X", _P), ("wq", _P), ("ws", _P), ("gscale", _F),
                ("wq2", _P), ("ws2", _P), ("gscale2", _F), ("out", _P), ("N", _I64), ("K", _I64)]


_SIGNATURES = {
    "nvfp4_packed_bytes": (_I, [_I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "nvfp4_pack_check": (_I, [_P, _P, _I64, _I64, _P, _P, _P]),
    "nvfp4_gemm_decode": (_I, [_P, _I, _P, _P, _F, _P, _I64, _I64, _P]),
    "nvfp4_gemm_decode_noalloc": (_I, [_P, _I, _P, _P, _F, _P, _I64, _I64, _P]),
    "nvfp4_gemm_gateup_silu": (_I, [_P, _I, _P, _P, _F, _P, _P, _F, _P, _I64, _I64, _P]),
    "nvfp4_round_create": (_I, [ctypes.POINTER(Nvfp4GemmDesc), _I, ctypes.POINTER(_P)]),
    "nvfp4_round_create_ex": (_I, [ctypes.POINTER(Nvfp4GemmDesc), _I, _I, ctypes.POINTER(_P)]),
    "nvfp4_round_nodes": (_I, [_P, ctypes.POINTER(_I)]),
    "nvfp4_round_replay": (_I, [_P, _I, _P]),
    "nvfp4_round_replay_host": (_I, [_P, _I, _P, _P, _SZ, _P, _P, _SZ, _P]),
    "nvfp4_round_destroy": (_I, [_P]),
    "nvfp4_topk": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _P]),
    "nvfp4_gemm_grouped": (_I, [_P, _I, _P, _I, _I, _P, _I, _P, _I64, _I64, _P]),
    "nvfp4_cache_fork": (_I, [ctypes.POINTER(Nvfp4Cache), _P, _P]),
    "nvfp4_cache_reserve": (_I, [ctypes.POINTER(Nvfp4Cache), _P, _P, _P]),
    "nvfp4_cache_compact": (_I, [ctypes.POINTER(Nvfp4Cache), _P, _P, _I, _P]),
    "nvfp4_cache_trim": (_I, [ctypes.POINTER(Nvfp4Cache), _P, _P]),
    "nvfp4_rope_append": (_I, [_P, _P]),
    "nvfp4_attn_tree": (_I, [_P, _P]),
    "nvfp4_attn_tree_workspace": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "nvfp4_beam_select": (_I, [_P, _I, _I, _I64, _I64, _P, _P, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "nvfp4_beam_select_workspace": (_I, [_I, _I, _I64, _I, ctypes.POINTER(_SZ)]),
    "nvfp4_topk_splits": (_I, [_I, _I64, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "nvfp4_verify_geometry": (_I, [_I, _I64, _I64, _I, ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                                   ctypes.POINTER(_I)]),
    "nvfp4_dequant_debug": (_I, [_P, _P, _F, _P, _I64, _I64, _P]),
    "nvfp4_unpack_debug": (_I, [_P, _P, _I64, _I64, _P, _P, _P]),
    "nvfp4_host_dequant_unit": (_I, [_P, _P, _F, _P]),
    "nvfp4_host_pack_unit": (_I, [_P, _P, _I64, _I64, _I64, _I64, _P, _P]),
    "nvfp4_stream_read": (_I, [_P, _SZ, _P, _I, _P]),
    "nvfp4_status_string": (ctypes.c_char_p, [_I]),
    "nvfp4_last_cuda_error": (_I, []),
    "nvfp4_device_status": (_I, []),
    "nvfp4_version": (_I, []),
}

_lib = None


def load():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def header_functions():
    """Names of the functions include/nvfp4decode.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"NVFP4_API\s+[\w\s\*]+?\b(nvfp4_\w+)\s*\(", text)))


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        msg = status_string(status)
        if status == NVFP4_ERR_CUDA:
            msg += f" (cuda error {load().nvfp4_last_cuda_error()})"
        super().__init__(f"{what}: {msg} [{status}]" if what else f"{msg} [{status}]")
        self.status = status


def status_string(status: int) -> str:
    return load().nvfp4_status_string(int(status)).decode()


def check(status: int, what: str = "") -> int:
    if status != NVFP4_OK:
        raise Nvfp4Error(status, what)
    return status


def _s(stream):
    return None if stream is None else int(stream)


# ------------------------------------------------------- raw C-ABI calls

def nvfp4_packed_bytes(N, K):
    """(status, wq_bytes, ws_bytes)."""
    a, b = _SZ(), _SZ()
    st = load().nvfp4_packed_bytes(int(N), int(K), ctypes.byref(a), ctypes.byref(b))
    return st, a.value, b.value


def nvfp4_pack_check(wq_canon, ws_canon, N, K, wq_dev, ws_dev, stream):
    return load().nvfp4_pack_check(wq_canon, ws_canon, int(N), int(K), wq_dev, ws_dev, _s(stream))


def nvfp4_gemm_decode(X, M, wq_dev, ws_dev, gscale, Y, N, K, stream):
    return load().nvfp4_gemm_decode(X, int(M), wq_dev, ws_dev, float(gscale), Y, int(N), int(K),
                                    _s(stream))


def nvfp4_gemm_decode_noalloc(X, M, wq_dev, ws_dev, gscale, Y, N, K, stream):
    """nvfp4_gemm_decode without any device allocation (static scratch array in the library)."""
    return load().nvfp4_gemm_decode_noalloc(X, int(M), wq_dev, ws_dev, float(gscale), Y, int(N), int(K),
                                            _s(stream))


def nvfp4_gemm_gateup_silu(X, M, wq_gate, ws_gate, gscale_gate, wq_up, ws_up, gscale_up, H, Nff, K,
                           stream):
    return load().nvfp4_gemm_gateup_silu(X, int(M), wq_gate, ws_gate, float(gscale_gate), wq_up,
                                         ws_up, float(gscale_up), H, int(Nff), int(K), _s(stream))


def nvfp4_round_create(descs):
    """(status, handle) for a sequence of Nvfp4GemmDesc."""
    arr = (Nvfp4GemmDesc * len(descs))(*descs)
    h = _P()
    st = load().nvfp4_round_create(arr, len(descs), ctypes.byref(h))
    return st, h.value


def nvfp4_round_create_ex(descs, mode):
    """(status, handle) for a sequence of Nvfp4GemmDesc, with a round mode."""
    arr = (Nvfp4GemmDesc * len(descs))(*descs)
    h = _P()
    st = load().nvfp4_round_create_ex(arr, len(descs), int(mode), ctypes.byref(h))
    return st, h.value


def nvfp4_round_nodes(handle):
    n = _I()
    st = load().nvfp4_round_nodes(handle, ctypes.byref(n))
    return st, n.value


def nvfp4_round_replay(handle, M, stream):
    return load().nvfp4_round_replay(handle, int(M), _s(stream))


def nvfp4_round_replay_host(handle, M, x_host, x_dev, x_bytes, y_dev, y_host, y_bytes, stream):
    return load().nvfp4_round_replay_host(handle, int(M), x_host, x_dev, int(x_bytes), y_dev, y_host,
                                          int(y_bytes), _s(stream))


def nvfp4_round_destroy(handle):
    return load().nvfp4_round_destroy(handle)


def nvfp4_gemm_grouped(X, x_per_route, route, M, T, experts, E, Y, N, K, stream):
    return load().nvfp4_gemm_grouped(X, int(x_per_route), route, int(M), int(T), experts, int(E), Y, int(N), int(K),
                                     _s(stream))


def nvfp4_cache_fork(cache, parent, stream):
    return load().nvfp4_cache_fork(cache, parent, _s(stream))


def nvfp4_cache_reserve(cache, want, ok, stream):
    return load().nvfp4_cache_reserve(cache, want, ok, _s(stream))


def nvfp4_cache_compact(cache, count, path, ld_path, stream):
    return load().nvfp4_cache_compact(cache, count, path, int(ld_path), _s(stream))


def nvfp4_cache_trim(cache, new_len, stream):
    return load().nvfp4_cache_trim(cache, new_len, _s(stream))


def nvfp4_rope_append(args, stream):
    """args: an Nvfp4RopeArgs by reference (ctypes.byref)."""
    return load().nvfp4_rope_append(args, _s(stream))


def nvfp4_attn_tree(args, stream):
    """args: an Nvfp4AttnArgs by reference (ctypes.byref)."""
    return load().nvfp4_attn_tree(args, _s(stream))


def nvfp4_attn_tree_workspace(rows, q_heads, kv_heads, head_dim, sm_count):
    """(status, bytes)."""
    n = _SZ()
    st = load().nvfp4_attn_tree_workspace(int(rows), int(q_heads), int(kv_heads), int(head_dim), int(sm_count),
                                          ctypes.byref(n))
    return st, n.value


def nvfp4_beam_select(logits, groups, beams, V, ldv, scores, finished, eos, scores_out, parent, token, finished_out,
                      workspace, workspace_bytes, stream):
    return load().nvfp4_beam_select(logits, int(groups), int(beams), int(V), int(ldv), scores, finished, int(eos),
                                    scores_out, parent, token, finished_out, workspace, int(workspace_bytes),
                                    _s(stream))


def nvfp4_beam_select_workspace(groups, beams, V, sm_count):
    """(status, bytes)."""
    n = _SZ()
    st = load().nvfp4_beam_select_workspace(int(groups), int(beams), int(V), int(sm_count), ctypes.byref(n))
    return st, n.value


def nvfp4_topk(logits, rows, V, ldv, k, values, indices, stream):
    return load().nvfp4_topk(logits, int(rows), int(V), int(ldv), int(k), values, indices, _s(stream))


def nvfp4_topk_splits(rows, V, k, sm_count):
    """(status, splits, slice) of the row split nvfp4_topk uses."""
    sp, sl = _I(0), _I(0)
    st = load().nvfp4_topk_splits(int(rows), int(V), int(k), int(sm_count), ctypes.byref(sp), ctypes.byref(sl))
    return st, sp.value, sl.value


def nvfp4_verify_geometry(M, N, K, sm_count):
    """(status, ctas, units, nl) of the verify-width work split."""
    c, u, nl = _I64(0), _I64(0), _I(0)
    st = load().nvfp4_verify_geometry(int(M), int(N), int(K), int(sm_count), ctypes.byref(c), ctypes.byref(u),
                                      ctypes.byref(nl))
    return st, c.value, u.value, nl.value


def nvfp4_dequant_debug(wq_dev, ws_dev, gscale, W, N, K, stream):
    return load().nvfp4_dequant_debug(wq_dev, ws_dev, float(gscale), W, int(N), int(K), _s(stream))


def nvfp4_unpack_debug(wq_dev, ws_dev, N, K, wq_canon, ws_canon, stream):
    return load().nvfp4_unpack_debug(wq_dev, ws_dev, int(N), int(K), wq_canon, ws_canon, _s(stream))


def nvfp4_host_dequant_unit(q_unit, s_unit, gscale, W):
    return load().nvfp4_host_dequant_unit(q_unit, s_unit, float(gscale), W)


def nvfp4_host_pack_unit(wq_canon, ws_canon, N, K, tile, chunk, q_unit, s_unit):
    return load().nvfp4_host_pack_unit(wq_canon, ws_canon, int(N), int(K), int(tile), int(chunk),
                                       q_unit, s_unit)


def nvfp4_stream_read(buf, nbytes, out, ctas, stream):
    return load().nvfp4_stream_read(buf, int(nbytes), out, int(ctas), _s(stream))


def nvfp4_status_string(status):
    return status_string(status)


def nvfp4_last_cuda_error():
    return load().nvfp4_last_cuda_error()


def nvfp4_device_status():
    return load().nvfp4_device_status()


def nvfp4_version():
    return load().nvfp4_version()


# ------------------------------------------------------- torch helpers

def _stream_ptr(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def pack(q_canon, s_canon, stream=None):
    """Pack canonical device planes (torch uint8 [N][K/2], [N][K/16]) into
    freshly allocated device-layout planes; returns (wq_dev, ws_dev)."""
    import torch
    N, half_k = q_canon.shape
    K = half_k * 2
    st, nq, ns = nvfp4_packed_bytes(N, K)
    check(st, "nvfp4_packed_bytes")
    wq = torch.empty(nq, dtype=torch.uint8, device=q_canon.device)
    ws = torch.empty(ns, dtype=torch.uint8, device=q_canon.device)
    check(nvfp4_pack_check(q_canon.data_ptr(), s_canon.data_ptr(), N, K, wq.data_ptr(),
                           ws.data_ptr(), _stream_ptr(stream)), "nvfp4_pack_check")
    return wq, ws


def gemm_decode(X, wq, ws, gscale, N, K, Y=None, stream=None):
    """Y float32 [M][N] = gscale * X . dequant(W)^T (X: torch bf16 [M][K] on the device)."""
    import torch
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    check(nvfp4_gemm_decode(X.data_ptr(), M, wq.data_ptr(), ws.data_ptr(), gscale, Y.data_ptr(), N,
                            K, _stream_ptr(stream)), "nvfp4_gemm_decode")
    return Y


def gemm_gateup_silu(X, wq_g, ws_g, gscale_g, wq_u, ws_u, gscale_u, Nff, K, H=None, stream=None):
    """H bf16 [M][Nff] = silu(X . Wg^T) * (X . Wu^T), one launch."""
    import torch
    M = X.shape[0]
    if H is None:
        H = torch.empty((M, Nff), dtype=torch.bfloat16, device=X.device)
    check(nvfp4_gemm_gateup_silu(X.data_ptr(), M, wq_g.data_ptr(), ws_g.data_ptr(), gscale_g,
                                 wq_u.data_ptr(), ws_u.data_ptr(), gscale_u, H.data_ptr(), Nff, K,
                                 _stream_ptr(stream)), "nvfp4_gemm_gateup_silu")
    return H


def expert_table(mats, device):
    """Device array of nvfp4_expert for a list of (wq, ws, gscale) device-layout planes."""
    import numpy as np
    import torch
    rec = np.zeros((len(mats), 3), dtype=np.uint64)
    for i, (wq, ws, gs) in enumerate(mats):
        rec[i, 0] = wq.data_ptr()
        rec[i, 1] = ws.data_ptr()
        rec[i, 2] = int(np.float32(gs).view(np.uint32))  # gscale in the low 32 bits, reserved = 0
    return torch.from_numpy(rec.view(np.int64)).to(device)


def gemm_grouped(X, route, experts, E, N, K, x_per_route=False, Y=None, stream=None):
    """Y float32 [M][T][N] for routes int32 [M][T] over the expert table (expert_table)."""
    import torch
    M, T = route.shape
    if Y is None:
        Y = torch.empty((M, T, N), dtype=torch.float32, device=X.device)
    check(nvfp4_gemm_grouped(X.data_ptr(), 1 if x_per_route else 0, route.data_ptr(), M, T, experts.data_ptr(), E,
                             Y.data_ptr(), N, K, _stream_ptr(stream)), "nvfp4_gemm_grouped")
    return Y


def topk(logits, k, V=None, values=None, indices=None, stream=None):
    """Top-k of each row of torch float32 [rows][ldv] device logits over the
    first V columns: (values float32 [rows][k], indices int32 [rows][k])."""
    import torch
    rows, ldv = logits.shape
    V = ldv if V is None else int(V)
    if logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    if values is None:
        values = torch.empty((rows, k), dtype=torch.float32, device=logits.device)
    if indices is None:
        indices = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    check(nvfp4_topk(logits.data_ptr(), rows, V, logits.stride(0), k, values.data_ptr(), indices.data_ptr(),
                     _stream_ptr(stream)), "nvfp4_topk")
    return values, indices


def _want(t, name, dtype, device, shape=None):
    """Raise unless `t` is a contiguous tensor of this dtype, device and shape; its pointer (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + (f" of shape {shape}" if shape else "") +
                         f" on {device}: got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _heads(t, name, dtype, device, heads, dim):
    """Check a [rows][heads][dim] or [rows][heads * dim] tensor whose rows are contiguous; (rows, row stride, pointer)."""
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}: got {t.dtype} on {t.device}")
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if not ((n == 2 and shape[1] == heads * dim and stride[1] == 1) or
            (n == 3 and shape[1] == heads and shape[2] == dim and stride[2] == 1 and
             (stride[1] == dim or heads == 1))):
        raise ValueError(f"{name} must be [rows][{heads}][{dim}] with contiguous rows: got {tuple(shape)} with "
                         f"strides {stride}")
    # a single row has no next one: its stride may be anything
    return shape[0], (stride[0] if shape[0] > 1 else heads * dim), t.data_ptr()


def _call(name, device, stream, *args):
    """The library's `name` with these arguments and a stream -- the device's current one, or the caller's -- with the
    device current; raises what its status says."""
    import torch
    index = device.index
    if stream is None:
        ptr = _current_stream(index)
    else:
        _same_device(stream, device)
        ptr = stream.cuda_stream
    fn = getattr(load(), name)
    if torch.cuda.current_device() == index:
        st = fn(*args, ptr)
    else:
        with torch.cuda.device(index):
            st = fn(*args, ptr)
    if st != NVFP4_OK:
        check(st, name)


def _same_device(stream, device):
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")


def _current_stream(index):
    """The current stream's handle on a device; without building a Stream object where torch allows (1.5 us a call)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


class Cache:
    """A paged cache of keys and values (nvfp4_cache): the tensors and the
    description the calls take.

    k, v: bfloat16 [layers][pages][kv_heads][page_size][head_dim]; table: int32
    [lanes][max_pages]; len: int32 [lanes]; ref: int32 [pages].  The tensors stay
    the caller's to read and to write between calls."""

    def __init__(self, k, v, table, len, ref):
        import torch
        dev = k.device
        if dev.type != "cuda":
            raise ValueError(f"the cache must be in device memory: got {dev}")
        if k.dim() != 5 or table.dim() != 2:
            raise ValueError("k and v must be [layers][pages][kv_heads][page_size][head_dim], table [lanes][max_pages]")
        layers, pages, heads, page, dim = k.shape
        lanes, width = table.shape
        i32 = torch.int32
        kp = _want(k, "k", torch.bfloat16, dev)
        vp = _want(v, "v", torch.bfloat16, dev, tuple(k.shape))
        tp = _want(table, "table", i32, dev)
        lp = _want(len, "len", i32, dev, (lanes,))
        rp = _want(ref, "ref", i32, dev, (pages,))
        self.k, self.v, self.table, self.len, self.ref = k, v, table, len, ref
        self.device, self.lanes, self.kv_heads, self.head_dim, self.page_size = dev, lanes, heads, dim, page
        self.scratch = torch.zeros(4 * lanes + 4, dtype=i32, device=dev)
        self.c = Nvfp4Cache(kp, vp, tp, lp, rp, self.scratch.data_ptr(), layers, pages, heads, page, dim, lanes, width, 0)
        self._ref = ctypes.byref(self.c)
        self._at = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, layers, pages, kv_heads, page_size, head_dim, lanes, max_pages, device):
        """A cache with every page free and every lane empty."""
        import torch
        shape = (layers, pages, kv_heads, page_size, head_dim)
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        i32 = torch.int32
        return cls(torch.zeros(shape, dtype=torch.bfloat16, device=dev),
                   torch.zeros(shape, dtype=torch.bfloat16, device=dev),
                   torch.full((lanes, max_pages), -1, dtype=i32, device=dev),
                   torch.zeros(lanes, dtype=i32, device=dev), torch.zeros(pages, dtype=i32, device=dev))

    def _lanes(self, t, name):
        import torch
        return _want(t, name, torch.int32, self.device, (self.lanes,))

    def fork(self, parent, stream=None):
        """Lane i takes lane parent[i]'s pages and length (-1: emptied)."""
        pp = self._lanes(parent, "parent")
        _call("nvfp4_cache_fork", self.device, stream, self._ref, pp)

    def reserve(self, want, ok=None, stream=None):
        """Room for want[b] more slots in each lane, in pages of its own: shared ones are copied or replaced.
        ok: int32 [1], set to 1 if every lane has its room, to 0 if not (too few free pages: nothing changes)."""
        import torch
        wp, op = self._lanes(want, "want"), _want(ok, "ok", torch.int32, self.device, (1,))
        _call("nvfp4_cache_reserve", self.device, stream, self._ref, wp, op)

    def compact(self, count, path=None, stream=None):
        """Commit count[b] drafted slots of each lane, those numbered path[b][:count[b]] (None: the first ones)."""
        import torch
        cp, pp, ld = self._lanes(count, "count"), None, 1
        if path is not None:
            pp = _want(path, "path", torch.int32, self.device)
            if path.dim() != 2 or path.shape[0] != self.lanes:
                raise ValueError(f"path must be [{self.lanes}][n]: got {tuple(path.shape)}")
            ld = path.shape[1]
        _call("nvfp4_cache_compact", self.device, stream, self._ref, cp, pp, ld)

    def trim(self, new_len, stream=None):
        """Cut lanes back to new_len[b] slots."""
        np_ = self._lanes(new_len, "new_len")
        _call("nvfp4_cache_trim", self.device, stream, self._ref, np_)


def _rope_record(cache, layer, y, q_heads, inv_freq, positions, pair_axis, style, row_start, q):
    """(nvfp4_rope_args as bytes, q) of a rotary append; see rope_append."""
    import torch
    dev, dim = cache.device, cache.head_dim
    rows, ldy, yp = _heads(y, "y", torch.float32, dev, q_heads + 2 * cache.kv_heads, dim)
    if q is None:
        q = torch.empty((rows, q_heads, dim), dtype=torch.bfloat16, device=dev)
    qrows, ldq, qp = _heads(q, "q", torch.bfloat16, dev, q_heads, dim)
    if qrows != rows:
        raise ValueError(f"q has {qrows} rows, y {rows}")
    half, axes, pp, fp = 0, 1, None, None
    if inv_freq is not None:
        half = inv_freq.shape[0]
        pp = _want(positions, "positions", torch.int32, dev)
        if positions is None or positions.dim() > 2 or positions.shape[-1] != rows:
            raise ValueError(f"positions must be [{rows}] or [axes][{rows}]")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        fp = _want(inv_freq, "inv_freq", torch.float64, dev, (half,))
    sp = _want(row_start, "row_start", torch.int32, dev, (cache.lanes + 1,))
    ap = _want(pair_axis, "pair_axis", torch.uint8, dev, (half,))
    return _ROPE_ARGS.pack(cache._at, layer, rows, q_heads, 2 * half, style, axes, yp, ldy, sp or 0, pp or 0, rows,
                           ap or 0, fp or 0, qp, ldq), q


def rope_append(cache, layer, y, q_heads, inv_freq, positions, pair_axis=None, style=NVFP4_ROPE_HALVES,
                row_start=None, q=None, stream=None):
    """Rotate the queries and keys of y (float32 [rows][(q_heads + 2 kv_heads) * head_dim], the q/k/v projection's
    output) and append keys and values to `layer` of the cache; returns q bfloat16 [rows][q_heads][head_dim].

    inv_freq: float64 [rot_dim / 2] (None: no rotation); positions: int32 [rows] or [axes][rows]; pair_axis: uint8
    [rot_dim / 2]; row_start: int32 [lanes + 1], or None for one row per lane."""
    if stream is not None:  # what is allocated here belongs to the stream that uses it
        import torch
        _same_device(stream, cache.device)
        with torch.cuda.stream(stream):
            return rope_append(cache, layer, y, q_heads, inv_freq, positions, pair_axis, style, row_start, q)
    a, q = _rope_record(cache, layer, y, q_heads, inv_freq, positions, pair_axis, style, row_start, q)
    _call("nvfp4_rope_append", cache.device, None, a)
    return q


_sms = {}


def _sm_count(device):
    import torch
    if device.index not in _sms:
        _sms[device.index] = torch.cuda.get_device_properties(device).multi_processor_count
    return _sms[device.index]


def attn_tree_workspace(cache, rows, q_heads):
    """A workspace for attn_tree calls of these sizes (uint8)."""
    import torch
    st, n = nvfp4_attn_tree_workspace(rows, q_heads, cache.kv_heads, cache.head_dim, _sm_count(cache.device))
    check(st, "nvfp4_attn_tree_workspace")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def _attn_record(cache, layer, q, scale, row_start, mask, max_nodes, out, want_lse, lse, workspace):
    """(nvfp4_attn_args as bytes, out, lse, workspace) of an attention call; see attn_tree."""
    import torch
    dev, dim = cache.device, cache.head_dim
    heads = q.shape[1] if q.dim() == 3 else q.shape[-1] // dim
    rows, ldq, qp = _heads(q, "q", torch.bfloat16, dev, heads, dim)
    if out is None:
        out = torch.empty_strided((rows, heads, dim), (heads * dim, dim, 1), dtype=torch.bfloat16, device=dev)
        ldo, op = heads * dim, out.data_ptr()
    else:
        orows, ldo, op = _heads(out, "out", torch.bfloat16, dev, heads, dim)
        if orows != rows:
            raise ValueError(f"out has {orows} rows, q {rows}")
    if lse is None and want_lse:
        lse = torch.empty_strided((rows, heads), (heads, 1), dtype=torch.float32, device=dev)
    sp = _want(row_start, "row_start", torch.int32, dev, (cache.lanes + 1,))
    mp = _want(mask, "mask", torch.int64, dev, (rows,))
    ep = _want(lse, "lse", torch.float32, dev, (rows, heads))
    if workspace is None:
        workspace = attn_tree_workspace(cache, rows, heads)
    wp = _want(workspace, "workspace", torch.uint8, dev)
    return _ATTN_ARGS.pack(cache._at, layer, rows, heads, max_nodes, scale, 0, qp, ldq, sp or 0, mp or 0, op, ldo,
                           ep or 0, wp, workspace.shape[0]), out, lse, workspace


def attn_tree(cache, layer, q, scale, row_start=None, mask=None, max_nodes=1, out=None, want_lse=False, lse=None,
              workspace=None, stream=None):
    """Attention of decode rows or drafted trees over `layer` of the cache: out bfloat16 [rows][q_heads][head_dim], or
    (out, lse float32 [rows][q_heads]) if lse is given or wanted.

    q: bfloat16 [rows][q_heads][head_dim]; row_start: int32 [lanes + 1], or None for one row per lane; mask: int64
    [rows], bit j of a row's word set where it sees its lane's j-th drafted slot (None: a chain); workspace: from
    attn_tree_workspace, one for each stream or graph whose calls may overlap (None: a new one)."""
    if stream is not None:  # what is allocated here belongs to the stream that uses it
        import torch
        _same_device(stream, cache.device)
        with torch.cuda.stream(stream):
            return attn_tree(cache, layer, q, scale, row_start, mask, max_nodes, out, want_lse, lse, workspace)
    a, out, lse, workspace = _attn_record(cache, layer, q, scale, row_start, mask, max_nodes, out, want_lse, lse,
                                          workspace)
    _call("nvfp4_attn_tree", cache.device, None, a)
    return out if lse is None else (out, lse)


def beam_select_workspace(groups, beams, vocab, device):
    """A zero-filled workspace for beam_select calls of these sizes (uint8)."""
    import torch
    st, n = nvfp4_beam_select_workspace(groups, beams, vocab, _sm_count(torch.device(device)))
    check(st, "nvfp4_beam_select_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def beam_select(logits, scores, vocab=None, finished=None, eos=-1, scores_out=None, parent=None, token=None,
                finished_out=None, workspace=None, stream=None):
    """The best continuations of each group of beams: (scores float32, parent int32, token int32, finished uint8), each
    [groups][beams], best first.

    logits: float32 [groups * beams][>= vocab], rows contiguous; scores: float32 [groups][beams]; finished: uint8
    [groups][beams] with its end token eos; parent is the row of logits that is extended (what Cache.fork takes)."""
    import torch
    if stream is not None:  # what is allocated here belongs to the stream that uses it
        _same_device(stream, logits.device)
        with torch.cuda.stream(stream):
            return beam_select(logits, scores, vocab, finished, eos, scores_out, parent, token, finished_out, workspace)
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError(f"logits must be in device memory: got {dev}")
    groups, beams = scores.shape
    size = logits.shape
    if len(size) != 2 or size[0] != groups * beams or logits.dtype is not torch.float32 or \
            (size[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be float32 [{groups * beams}][vocab] with contiguous rows")
    V = size[1] if vocab is None else int(vocab)
    if V > size[1]:
        raise ValueError(f"vocab {V} is past the logits' {size[1]} columns")
    # a single row has no next one: its stride may be anything
    ldv = logits.stride(0) if size[0] > 1 else (V + 3) // 4 * 4
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    shape = (groups, beams)
    sp = _want(scores, "scores", f32, dev, shape)
    # (what is allocated here needs no check: 0.5 us each)
    if scores_out is None:
        scores_out = torch.empty_like(scores)
        op = scores_out.data_ptr()
    else:
        op = _want(scores_out, "scores_out", f32, dev, shape)
    if parent is None:
        parent = torch.empty_like(scores, dtype=i32)
        pp = parent.data_ptr()
    else:
        pp = _want(parent, "parent", i32, dev, shape)
    if token is None:
        token = torch.empty_like(scores, dtype=i32)
        tp = token.data_ptr()
    else:
        tp = _want(token, "token", i32, dev, shape)
    if finished_out is None:
        finished_out = torch.empty_like(scores, dtype=u8)
        dp = finished_out.data_ptr()
    else:
        dp = _want(finished_out, "finished_out", u8, dev, shape)
    if workspace is None:
        workspace = beam_select_workspace(groups, beams, V, dev)
    _call("nvfp4_beam_select", dev, None, logits.data_ptr(), groups, beams, V, ldv, sp,
          _want(finished, "finished", u8, dev, shape), eos, op, pp, tp, dp, _want(workspace, "workspace", u8, dev),
          workspace.shape[0])
    return scores_out, parent, token, finished_out


def stream_read(buf, ctas, out=None, stream=None):
    """Read every byte of the contiguous device tensor `buf` once (nvfp4_stream_read);
    returns the uint32 [ctas] device tensor of per-CTA XORs (as int32)."""
    import torch
    if not buf.is_contiguous():
        raise ValueError("buf must be contiguous")
    if out is None:
        out = torch.empty((ctas,), dtype=torch.int32, device=buf.device)
    check(nvfp4_stream_read(buf.data_ptr(), buf.numel() * buf.element_size(), out.data_ptr(), ctas,
                            _stream_ptr(stream)), "nvfp4_stream_read")
    return out


def dequant_debug(wq, ws, gscale, N, K, stream=None):
    import torch
    W = torch.empty((N, K), dtype=torch.float32, device=wq.device)
    check(nvfp4_dequant_debug(wq.data_ptr(), ws.data_ptr(), gscale, W.data_ptr(), N, K,
                              _stream_ptr(stream)), "nvfp4_dequant_debug")
    return W


def unpack_debug(wq, ws, N, K, stream=None):
    import torch
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=wq.device)
    s = torch.empty((N, K // 16), dtype=torch.uint8, device=wq.device)
    check(nvfp4_unpack_debug(wq.data_ptr(), ws.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
                             _stream_ptr(stream)), "nvfp4_unpack_debug")
    return q, s


class Round:
    """Owner of an nvfp4_round handle built from descriptors."""

    def __init__(self, descs, mode=None):
        if mode is None:
            st, h = nvfp4_round_create(descs)
        else:
            st, h = nvfp4_round_create_ex(descs, mode)
        check(st, "nvfp4_round_create")
        self.handle = h
        self._descs = list(descs)

    @property
    def nodes(self):
        st, n = nvfp4_round_nodes(self.handle)
        check(st, "nvfp4_round_nodes")
        return n

    def replay(self, M, stream=None):
        check(nvfp4_round_replay(self.handle, M, _stream_ptr(stream)), "nvfp4_round_replay")

    def replay_host(self, M, x_host, x_dev, y_dev, y_host, stream=None):
        """H2D copy of x_host -> x_dev, replay, D2H copy of y_dev -> y_host (torch tensors)."""
        xb = x_host.numel() * x_host.element_size()
        yb = y_host.numel() * y_host.element_size()
        check(nvfp4_round_replay_host(self.handle, M, x_host.data_ptr(), x_dev.data_ptr(), xb,
                                      y_dev.data_ptr(), y_host.data_ptr(), yb, _stream_ptr(stream)),
              "nvfp4_round_replay_host")

    def close(self):
        if self.handle:
            nvfp4_round_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def desc(kind, X, wq, ws, gscale, out, N, K, wq2=None, ws2=None, gscale2=0.0):
    """An Nvfp4GemmDesc from torch tensors."""
    return Nvfp4GemmDesc(kind, X.data_ptr(), wq.data_ptr(), ws.data_ptr(), float(gscale),
                         wq2.data_ptr() if wq2 is not None else None,
                         ws2.data_ptr() if ws2 is not None else None, float(gscale2),
                         out.data_ptr(), int(N), int(K))


def _between(kind, record, *keep):
    """A descriptor whose X is the record (kept alive with the tensors it names for as long as the descriptor)."""
    buf = ctypes.create_string_buffer(record, len(record))
    d = Nvfp4GemmDesc(kind, ctypes.addressof(buf))
    d._keep = (buf, *keep)
    return d


def _round_rows(t, name):
    """A round keeps the tensor's address and runs at widths of up to 8 rows: it is the caller's, and has them all."""
    if t is None:
        raise ValueError(f"{name} must be given: a round's nodes keep its address")
    if t.dim() < 2 or t.shape[0] < NVFP4_ROUND_ROWS:
        raise ValueError(f"{name} must have {NVFP4_ROUND_ROWS} rows, the widest round's: got {tuple(t.shape)}")


def desc_rope(cache, layer, y, q_heads, inv_freq, positions, q, pair_axis=None, style=NVFP4_ROPE_HALVES):
    """An Nvfp4GemmDesc of a round's rotary append: rope_append's arguments with one row per lane, 8 rows, q given.  The
    tensors are kept with the descriptor and must outlive the round."""
    _round_rows(y, "y")
    _round_rows(q, "q")
    record, _ = _rope_record(cache, layer, y, q_heads, inv_freq, positions, pair_axis, style, None, q)
    return _between(NVFP4_DESC_ROPE_APPEND, record, cache, y, inv_freq, positions, q, pair_axis)


def desc_attn(cache, layer, q, scale, out, workspace, lse=None):
    """An Nvfp4GemmDesc of a round's attention: attn_tree's arguments with one row per lane, 8 rows, out and workspace
    given.  The tensors are kept with the descriptor and must outlive the round."""
    _round_rows(q, "q")
    _round_rows(out, "out")
    if workspace is None:
        raise ValueError("workspace must be given: a round's nodes keep its address")
    record = _attn_record(cache, layer, q, scale, None, None, 1, out, False, lse, workspace)[0]
    return _between(NVFP4_DESC_ATTN_TREE, record, cache, q, out, workspace, lse)
