"""Python binding of libw4q.so (include/w4q.h): argument marshalling only.

Every function takes torch CUDA tensors, checks dtype / shape / contiguity,
allocates outputs and workspace with torch when the caller passes none, and
calls the C entry point of the same name on the current CUDA stream.  All
arithmetic happens in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw4q.so")
GROUP = 32

_lib = None
_lock = threading.Lock()

W4Q_OK = 0
STATUS = {
    0: "W4Q_OK", 1: "W4Q_ERR_INVALID_ARG", 2: "W4Q_ERR_UNSUPPORTED", 3: "W4Q_ERR_MISALIGNED",
    4: "W4Q_ERR_WORKSPACE", 5: "W4Q_ERR_CUDA", 6: "W4Q_ERR_DEVICE",
}

# name -> (restype, argtypes) for every symbol of include/w4q.h
_P, _I64, _INT, _SZ, _U32P = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                              ctypes.POINTER(ctypes.c_uint32))
_F = ctypes.c_float
SIGNATURES = {
    "w4q_status_string": (ctypes.c_char_p, [_INT]),
    "w4_packed_bytes": (_SZ, [_I64, _I64, _INT]),
    "w4_pack_weights": (_INT, [_P, _I64, _I64, _INT, _P, _P]),
    "w4_unpack_weights": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P, _P]),
    "w4_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "w4_workspace_bytes_split": (_SZ, [_I64, _I64, _I64, _INT, _INT]),
    "w4_split_choice": (_INT, [_I64, _I64, _I64, _INT]),
    "w4_kernel_launches": (_INT, [_I64, _I64, _I64, _INT, _INT]),
    "w4a16_gemm": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]),
    "w4a16_gemm_split": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _INT, _P, _SZ, _P]),
    "w4a16_gemm_noalloc": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _P]),
    "w4a8_gemm": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]),
    "w4a8_gemm_split": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _INT, _P, _SZ, _P]),
    "w4a8_quantize_act": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "w4a8_group_dots": (_INT, [_P, _P, _I64, _I64, _I64, _INT, _P, _P, _SZ, _P]),
    "w4a8_gemm_rowscale": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _P, _SZ, _P]),
    "w4a8_gemm_rowscale_split": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _INT, _P, _SZ, _P]),
    "w4a8_quantize_act_rowscale": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "w4a8_group_dots_rowscale": (_INT, [_P, _P, _I64, _I64, _I64, _INT, _P, _P, _SZ, _P]),
    "w8_gemv": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w8_gemm": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "w8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "w8_kernel_launches": (_INT, [_I64, _I64, _I64]),
    "w4_packed_bytes_compact": (_SZ, [_I64, _I64, _INT]),
    "w4_pack_weights_compact": (_INT, [_P, _I64, _I64, _INT, _P, _P]),
    "w4_unpack_weights_compact": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P, _P, _P]),
    "w4a16_gemm_compact": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, _P]),
    "qk_norm_rope": (_INT, [_P, _P, _I64, _INT, _INT, _INT, _I64, _I64, _P, _P, _F, _P, _I64, _INT,
                            _INT, _P, _P, _P, _P]),
    "kv8_append": (_INT, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _I64, _INT, _P, _P, _P, _F, _P, _I64,
                          _INT, _INT, _P]),
    "kv8_read": (_INT, [_P, _P, _I64, _P, _P, _P]),
    "kv8_attention": (_INT, [_P, _P, _I64, _P, _P, _INT, _INT, _F, _I64, _P, _SZ, _P]),
    "moe_w4a16": (_INT, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _INT, _INT, _INT, _F, _P, _P,
                         _P, _SZ, _P]),
    "moe_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _INT]),
    "kv8_workspace_bytes": (_SZ, [_I64, _INT, _INT, _INT, _INT]),
    "w4q_device_error": (_INT, [_U32P]),
    "w4q_selftest_wait_expiry": (_INT, [ctypes.c_uint, _P]),
}


class W4QError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s" % (fn, STATUS.get(status, status)))


def lib():
    """The loaded libw4q.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libw4q.so is not built (run __graft_entry__.build() or "
                                   "python gemv_w4a16_gemm_gb300/build.py)")
            l = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(l, name)
                fn.restype = res
                fn.argtypes = args
            _lib = l
    return _lib


def _check(fn: str, status: int):
    if status != W4Q_OK:
        raise W4QError(fn, status)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _cuda(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def status_string(status: int) -> str:
    return lib().w4q_status_string(status).decode()


def packed_bytes(N: int, K: int, group: int = GROUP) -> int:
    return int(lib().w4_packed_bytes(N, K, group))


def workspace_bytes(M: int, N: int, K: int, group: int = GROUP, split_k: int | None = None) -> int:
    if split_k is None:
        return int(lib().w4_workspace_bytes(M, N, K, group))
    return int(lib().w4_workspace_bytes_split(M, N, K, group, split_k))


def split_choice(M: int, N: int, K: int, group: int = GROUP) -> int:
    return int(lib().w4_split_choice(M, N, K, group))


def kernel_launches(M: int, N: int, K: int, w4a8=False, group: int = GROUP) -> int:
    """Kernels one call launches: w4a8 False = W4A16, True or "group" = W4A8
    with a scale per group of 32, "row" = W4A8 with a scale per row."""
    mode = 2 if w4a8 == "row" else (1 if w4a8 else 0)
    return int(lib().w4_kernel_launches(M, N, K, group, mode))


def _workspace(M, N, K, group, split_k, workspace, device):
    # a given workspace is passed as is (the library checks its size)
    if workspace is None:
        need = workspace_bytes(M, N, K, group, split_k)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def w4_pack_weights(W: torch.Tensor, group: int = GROUP, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """bf16 [N,K] CUDA weight -> packed uint8 buffer (layout of include/w4q.h)."""
    N, K = W.shape
    pw = _cuda(W, torch.bfloat16, "W")
    nbytes = packed_bytes(N, K, group)
    if nbytes == 0:
        raise W4QError("w4_pack_weights", 2)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    po = _cuda(out, torch.uint8, "out")
    _check("w4_pack_weights", lib().w4_pack_weights(pw, N, K, group, po, _stream(stream)))
    return out


def w4_unpack_weights(packed: torch.Tensor, N: int, K: int, group: int = GROUP, stream=None):
    """packed -> (q u8 [N,K], scale bf16 [N,K/32], zero u8 [N,K/32])."""
    dev = packed.device
    q = torch.empty(N, K, dtype=torch.uint8, device=dev)
    s = torch.empty(N, K // group, dtype=torch.bfloat16, device=dev)
    z = torch.empty(N, K // group, dtype=torch.uint8, device=dev)
    _check("w4_unpack_weights", lib().w4_unpack_weights(
        _cuda(packed, torch.uint8, "packed"), N, K, group, q.data_ptr(), s.data_ptr(),
        z.data_ptr(), _stream(stream)))
    return q, s, z


def _gemm(name, x, packed, N, K, group, split_k, out, workspace, stream):
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be [M, %d]" % K)
    px = _cuda(x, torch.bfloat16, "x")
    pp = _cuda(packed, torch.uint8, "packed")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    po = _cuda(out, torch.bfloat16, "out")
    ws, wsb = _workspace(M, N, K, group, split_k, workspace, x.device)
    pws = _cuda(ws, ws.dtype, "workspace")
    l = lib()
    if split_k is None:
        st = getattr(l, name)(px, pp, po, M, N, K, group, pws, wsb, _stream(stream))
    else:
        st = getattr(l, name + "_split")(px, pp, po, M, N, K, group, split_k, pws, wsb,
                                         _stream(stream))
    _check(name, st)
    return out


def w4a16_gemm(x, packed, N, K, group=GROUP, split_k=None, out=None, workspace=None, stream=None):
    """out[M,N] = x . dequant(packed)^T (W4A16); split_k None = library choice."""
    return _gemm("w4a16_gemm", x, packed, N, K, group, split_k, out, workspace, stream)


def w4a16_gemm_noalloc(x, packed, N, K, group=GROUP, out=None, stream=None):
    """W4A16 without any workspace: the library's own static scratch array is
    used (for callers that cannot allocate; see include/w4q.h)."""
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be [M, %d]" % K)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    _check("w4a16_gemm_noalloc", lib().w4a16_gemm_noalloc(
        _cuda(x, torch.bfloat16, "x"), _cuda(packed, torch.uint8, "packed"),
        _cuda(out, torch.bfloat16, "out"), M, N, K, group, _stream(stream)))
    return out


def w4a8_gemm(x, packed, N, K, group=GROUP, split_k=None, out=None, workspace=None, stream=None):
    """out[M,N] = x . dequant(packed)^T, W4A8 with one int8 activation scale
    per (row, group of 32)."""
    return _gemm("w4a8_gemm", x, packed, N, K, group, split_k, out, workspace, stream)


def w4a8_gemm_rowscale(x, packed, N, K, group=GROUP, split_k=None, out=None, workspace=None,
                       stream=None):
    """out[M,N] = x . dequant(packed)^T, W4A8 with one int8 activation scale
    per row (absmax / 127)."""
    return _gemm("w4a8_gemm_rowscale", x, packed, N, K, group, split_k, out, workspace, stream)


def _quantize_act(name, x, row, stream):
    M, K = x.shape
    xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
    sx = torch.empty((M,) if row else (M, K // GROUP), dtype=torch.float32, device=x.device)
    _check(name, getattr(lib(), name)(
        _cuda(x, torch.bfloat16, "x"), M, K, xq.data_ptr(), sx.data_ptr(), _stream(stream)))
    return xq, sx


def w4a8_quantize_act(x: torch.Tensor, stream=None):
    """(xq int8 [M,K], sx fp32 [M, K/32]): the per-group W4A8 quantizer."""
    return _quantize_act("w4a8_quantize_act", x, False, stream)


def w4a8_quantize_act_rowscale(x: torch.Tensor, stream=None):
    """(xq int8 [M,K], sx fp32 [M]): the per-row W4A8 quantizer."""
    return _quantize_act("w4a8_quantize_act_rowscale", x, True, stream)


def _group_dots(name, x, packed, N, K, group, workspace, stream):
    M = x.shape[0]
    D = torch.empty(M, N, K // group, dtype=torch.int32, device=x.device)
    ws, wsb = _workspace(M, N, K, group, None, workspace, x.device)
    _check(name, getattr(lib(), name)(
        _cuda(x, torch.bfloat16, "x"), _cuda(packed, torch.uint8, "packed"), M, N, K, group,
        D.data_ptr(), ws.data_ptr(), wsb, _stream(stream)))
    return D


def w4a8_group_dots(x, packed, N, K, group=GROUP, workspace=None, stream=None):
    """Exact int32 W4A8 group dots [M, N, K/32] (per-group activation scales)."""
    return _group_dots("w4a8_group_dots", x, packed, N, K, group, workspace, stream)


def w4a8_group_dots_rowscale(x, packed, N, K, group=GROUP, workspace=None, stream=None):
    """Exact int32 W4A8 group dots [M, N, K/32] (per-row activation scales)."""
    return _group_dots("w4a8_group_dots_rowscale", x, packed, N, K, group, workspace, stream)


def packed_bytes_compact(N: int, K: int, group: int = GROUP) -> int:
    return int(lib().w4_packed_bytes_compact(N, K, group))


def w4_pack_weights_compact(W: torch.Tensor, group: int = GROUP, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """bf16 [N,K] CUDA weight -> packed uint8 buffer with the compact metadata
    (uint8 scale / zero codes, fp16 row steps; layout of include/w4q.h)."""
    N, K = W.shape
    pw = _cuda(W, torch.bfloat16, "W")
    nbytes = packed_bytes_compact(N, K, group)
    if nbytes == 0:
        raise W4QError("w4_pack_weights_compact", 2)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    po = _cuda(out, torch.uint8, "out")
    _check("w4_pack_weights_compact",
           lib().w4_pack_weights_compact(pw, N, K, group, po, _stream(stream)))
    return out


def w4_unpack_weights_compact(packed: torch.Tensor, N: int, K: int, group: int = GROUP,
                              stream=None):
    """packed -> (q u8 [N,K], scale codes u8 [N,K/32], zero codes u8 [N,K/32],
    steps fp16 [N,2])."""
    dev = packed.device
    q = torch.empty(N, K, dtype=torch.uint8, device=dev)
    sc = torch.empty(N, K // group, dtype=torch.uint8, device=dev)
    zc = torch.empty(N, K // group, dtype=torch.uint8, device=dev)
    st = torch.empty(N, 2, dtype=torch.float16, device=dev)
    _check("w4_unpack_weights_compact", lib().w4_unpack_weights_compact(
        _cuda(packed, torch.uint8, "packed"), N, K, group, q.data_ptr(), sc.data_ptr(),
        zc.data_ptr(), st.data_ptr(), _stream(stream)))
    return q, sc, zc, st


def w4a16_gemm_compact(x, packed, N, K, group=GROUP, out=None, stream=None):
    """out[M,N] = x . dequant(packed)^T with the compact metadata (M <= 8)."""
    M = x.shape[0]
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be [M, %d]" % K)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    _check("w4a16_gemm_compact", lib().w4a16_gemm_compact(
        _cuda(x, torch.bfloat16, "x"), _cuda(packed, torch.uint8, "packed"),
        _cuda(out, torch.bfloat16, "out"), M, N, K, group, _stream(stream)))
    return out


def w8_gemv(x, W, scales, out=None, stream=None):
    """out[M,N] = bf16((x . W^T) * scales), int8 W [N,K], bf16 scales [N]."""
    M, K = x.shape
    N = W.shape[0]
    px = _cuda(x, torch.bfloat16, "x")
    pw = _cuda(W, torch.int8, "W")
    ps = _cuda(scales, torch.bfloat16, "scales")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    po = _cuda(out, torch.bfloat16, "out")
    _check("w8_gemv", lib().w8_gemv(px, pw, ps, po, M, N, K, _stream(stream)))
    return out


def w8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().w8_workspace_bytes(M, N, K))


def w8_kernel_launches(M: int, N: int, K: int) -> int:
    return int(lib().w8_kernel_launches(M, N, K))


def w8_gemm(x, W, scales, out=None, workspace=None, stream=None):
    """w8_gemv for 1 <= M <= 64 (the tensor-core path needs a workspace;
    one is allocated when none is given)."""
    M, K = x.shape
    N = W.shape[0]
    px = _cuda(x, torch.bfloat16, "x")
    pw = _cuda(W, torch.int8, "W")
    ps = _cuda(scales, torch.bfloat16, "scales")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    po = _cuda(out, torch.bfloat16, "out")
    need = w8_workspace_bytes(M, N, K)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    pws = _cuda(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check("w8_gemm", lib().w8_gemm(px, pw, ps, po, M, N, K, pws, nbytes, _stream(stream)))
    return out


# ------------------------------------------------ between the linear layers

class _Kv8Cache(ctypes.Structure):
    """w4q_kv8_cache of include/w4q.h."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("block_table", _P),
                ("seq_lens", _P), ("blocks", _I64), ("seqs", ctypes.c_int32),
                ("width", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page", ctypes.c_int32), ("format", ctypes.c_int32)]


def _new(make, shape, dtype, device, stream):
    """make(shape) (torch.empty or torch.zeros) on the stream that the call
    runs on, so that its memory belongs to that stream and a fill comes first."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _heads(t: torch.Tensor, name: str, tokens=None, heads=None, dim=None):
    """(pointer, row stride) of head rows bf16 [tokens, heads, head_dim]: a
    token's heads lie one after the other, tokens may lie further apart."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != torch.bfloat16 or t.dim() != 3:
        raise ValueError("%s must be bfloat16 [tokens, heads, head_dim]" % name)
    n, h, d = t.shape
    if (tokens is not None and n != tokens) or (heads is not None and h != heads) or \
            (dim is not None and d != dim):
        raise ValueError("%s must be [%s, %s, %s], got %s" % (
            name, "*" if tokens is None else tokens, "*" if heads is None else heads,
            "*" if dim is None else dim, tuple(t.shape)))
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError("a token's heads must lie one after the other in %s" % name)
    return t.data_ptr(), s0 if n > 1 else h * d


def _optional(t, dtype, name, numel=None):
    if t is None:
        return None
    p = _cuda(t, dtype, name)
    if numel is not None and t.numel() != numel:
        raise ValueError("%s must have %d elements, got %d" % (name, numel, t.numel()))
    return p


def _table(cos_sin):
    if cos_sin is None:
        return None, 0, 0
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rot]")
    return _cuda(cos_sin, torch.float32, "cos_sin"), cos_sin.shape[0], cos_sin.shape[1]


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """(q, k) normed per head and rotated, bf16 [tokens, heads, head_dim]
    (k may be None).  cos_sin: fp32 [positions, rot], the cosines of the
    rot / 2 angles of a position, then the sines; positions: int32 [tokens]."""
    pq, sq = _heads(q, "q")
    n, hq, d = q.shape
    pk, sk, hk = None, 0, 0
    if k is not None:
        pk, sk = _heads(k, "k", n, None, d)
        hk = k.shape[1]
    pt, npos, rot = _table(cos_sin)
    if q_out is None:
        q_out = _new(torch.empty, (n, hq, d), torch.bfloat16, q.device, stream)
    po = _optional(q_out, torch.bfloat16, "q_out", n * hq * d)
    if k is not None and k_out is None:
        k_out = _new(torch.empty, (n, hk, d), torch.bfloat16, q.device, stream)
    pko = _optional(k_out, torch.bfloat16, "k_out", n * hk * d)
    _check("qk_norm_rope", lib().qk_norm_rope(
        pq, pk, n, hq, hk, d, sq, sk, _optional(q_weight, torch.bfloat16, "q_weight", d),
        _optional(k_weight, torch.bfloat16, "k_weight", d), eps, pt, npos, rot, bool(interleaved),
        _optional(positions, torch.int32, "positions", n), po, pko, _stream(stream)))
    return q_out, k_out


def _kv8(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens):
    blocks, kv_heads, page, d = k_cache.shape
    if k_cache.dtype not in (torch.int8, torch.float8_e4m3fn):
        raise ValueError("k_cache must be int8 or float8_e4m3fn, got %s" % k_cache.dtype)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    if block_table.dim() != 2 or seq_lens.dim() != 1 or block_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("block_table must be [seqs, width], seq_lens [seqs]")
    n = blocks * kv_heads
    return _Kv8Cache(
        _cuda(k_cache, k_cache.dtype, "k_cache"), _cuda(v_cache, k_cache.dtype, "v_cache"),
        _optional(k_scale, torch.float32, "k_scale", n), _optional(v_scale, torch.float32, "v_scale", n),
        _cuda(block_table, torch.int32, "block_table"), _cuda(seq_lens, torch.int32, "seq_lens"),
        blocks, block_table.shape[0], block_table.shape[1], kv_heads, d, page,
        0 if k_cache.dtype == torch.int8 else 1)


def _cu(cu_tokens, seqs):
    return _optional(cu_tokens, torch.int32, "cu_tokens", seqs + 1)


def kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_tokens=None,
               q=None, q_out=None, q_weight=None, k_weight=None, cos_sin=None, eps=1e-6,
               interleaved=False, stream=None):
    """Write the step's keys and values bf16 [tokens, kv_heads, head_dim] into
    the 8-bit cache (k_cache, v_cache: int8 or float8_e4m3fn [blocks,
    kv_heads, page, head_dim]; scales fp32 [blocks, kv_heads]), the keys normed
    and rotated first where k_weight / cos_sin are given.  seq_lens counts the
    new tokens; cu_tokens int32 [seqs + 1], or None: one token each.  With q,
    returns the queries normed and rotated too (q_out), else None."""
    c = _kv8(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    n, d = k.shape[0], c.head_dim
    pk, sk = _heads(k, "k", None, c.kv_heads, d)
    pv, sv = _heads(v, "v", n, c.kv_heads, d)
    pq, sq, hq, po = None, 0, 0, None
    if q is not None:
        pq, sq = _heads(q, "q", n, None, d)
        hq = q.shape[1]
        if q_out is None:
            q_out = _new(torch.empty, (n, hq, d), torch.bfloat16, q.device, stream)
        po = _optional(q_out, torch.bfloat16, "q_out", n * hq * d)
    pt, npos, rot = _table(cos_sin)
    _check("kv8_append", lib().kv8_append(
        ctypes.byref(c), pk, pv, sk, sv, n, _cu(cu_tokens, c.seqs), pq, sq, hq, po,
        _optional(q_weight, torch.bfloat16, "q_weight", d),
        _optional(k_weight, torch.bfloat16, "k_weight", d), eps, pt, npos, rot, bool(interleaved),
        _stream(stream)))
    return q_out


def kv8_read(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_tokens=None, tokens=None,
             stream=None):
    """(k, v) bf16 [tokens, kv_heads, head_dim]: what the cache holds of the
    last cu_tokens[b + 1] - cu_tokens[b] positions of each sequence (None: the
    last one).  tokens: cu_tokens' last value, known on the host."""
    c = _kv8(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    if tokens is None:
        if cu_tokens is not None:
            raise ValueError("tokens must be given with cu_tokens")
        tokens = c.seqs
    k = _new(torch.empty, (tokens, c.kv_heads, c.head_dim), torch.bfloat16, k_cache.device, stream)
    v = _new(torch.empty, k.shape, torch.bfloat16, k_cache.device, stream)
    _check("kv8_read", lib().kv8_read(ctypes.byref(c), _cu(cu_tokens, c.seqs), tokens, k.data_ptr(),
                                      v.data_ptr(), _stream(stream)))
    return k, v


def kv8_workspace_bytes(seqs: int, queries: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().kv8_workspace_bytes(seqs, queries, heads, kv_heads, head_dim))


def kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale=None,
                  window=0, out=None, lse=None, workspace=None, stream=None):
    """Attention of q bf16 [seqs, queries, heads, head_dim], the last tokens of
    their sequences, over the 8-bit cache; scale None: head_dim ** -0.5.
    window > 0: each query sees the last `window` positions up to its own.
    lse: fp32 [seqs, queries, heads] to be written, or None.  workspace:
    kv8_workspace_bytes bytes, zero before the first use (one is made if it is
    None)."""
    c = _kv8(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    if q.dim() != 4 or q.shape[0] != c.seqs or q.shape[3] != c.head_dim:
        raise ValueError("q must be [%d, queries, heads, %d]" % (c.seqs, c.head_dim))
    n, m, hq, d = q.shape
    if n > 1 and m > 1 and q.stride(0) != m * q.stride(1):
        raise ValueError("the query tokens must lie at one stride in q")
    pq, sq = _heads(q[:, 0] if m == 1 else q.flatten(0, 1), "q")
    if out is None:
        out = _new(torch.empty, (n, m, hq, d), torch.bfloat16, q.device, stream)
    po = _optional(out, torch.bfloat16, "out", n * m * hq * d)
    if workspace is None:
        workspace = _new(torch.zeros, (max(16, kv8_workspace_bytes(n, m, hq, c.kv_heads, d)),), torch.uint8,
                         q.device, stream)
    _check("kv8_attention", lib().kv8_attention(
        ctypes.byref(c), pq, sq, po, _optional(lse, torch.float32, "lse", n * m * hq), m, hq,
        d ** -0.5 if scale is None else scale, window, _cuda(workspace, workspace.dtype, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def moe_workspace_bytes(tokens: int, hidden: int, inter: int, experts: int, topk: int) -> int:
    return int(lib().moe_workspace_bytes(tokens, hidden, inter, experts, topk))


def moe_w4a16(x, router, w13, w2, inter, topk, bias=None, sigmoid=False, renormalize=True, scale=1.0,
              out=None, ids=None, weights=None, workspace=None, stream=None):
    """A mixture-of-experts layer for x bf16 [tokens, hidden] (1..64 tokens):
    router bf16 [experts, hidden]; w13 = w4_pack_weights of [experts * 2 *
    inter, hidden] (an expert's gate rows, then its up rows); w2 =
    w4_pack_weights of [experts * hidden, inter].  sigmoid: sigmoid scores, the
    choice by score + bias (fp32 [experts] or None); else softmax.  ids, weights:
    int32 / fp32 [tokens, topk] to be written, or None."""
    if x.dim() != 2 or router.dim() != 2 or router.shape[1] != x.shape[1]:
        raise ValueError("x must be [tokens, hidden], router [experts, hidden]")
    m, h = x.shape
    e = router.shape[0]
    px, pr = _cuda(x, torch.bfloat16, "x"), _cuda(router, torch.bfloat16, "router")
    p13, p2 = _cuda(w13, torch.uint8, "w13"), _cuda(w2, torch.uint8, "w2")
    if w13.numel() != packed_bytes(e * 2 * inter, h) or w2.numel() != packed_bytes(e * h, inter):
        raise ValueError("w13 and w2 must be packed from [%d, %d] and [%d, %d]" % (e * 2 * inter, h, e * h, inter))
    if out is None:
        out = _new(torch.empty, (m, h), torch.bfloat16, x.device, stream)
    if workspace is None:
        workspace = _new(torch.empty, (max(16, moe_workspace_bytes(m, h, inter, e, topk)),), torch.uint8,
                         x.device, stream)
    _check("moe_w4a16", lib().moe_w4a16(
        px, pr, _optional(bias, torch.float32, "bias", e), p13, p2, _optional(out, torch.bfloat16, "out", m * h),
        m, h, inter, e, topk, bool(sigmoid), bool(renormalize), scale,
        _optional(ids, torch.int32, "ids", m * topk), _optional(weights, torch.float32, "weights", m * topk),
        _cuda(workspace, workspace.dtype, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


def device_error() -> int:
    """Read and clear the device-side error word (synchronizes)."""
    v = ctypes.c_uint32(0)
    st = lib().w4q_device_error(ctypes.byref(v))
    if st not in (W4Q_OK, 6):
        raise W4QError("w4q_device_error", st)
    return int(v.value)
