"""qlin: quantized linear layers for AMD Instinct MI355X (gfx950).

Thin Python binding over the C ABI of ``libqlin.so`` (``include/qlin.h``).
Every computation runs in the library's HIP kernels; this module only checks
tensors, allocates outputs with torch and passes raw device pointers plus
the current HIP stream. Importing it fails loudly if the library has not been
built (``python quantized_linear_layers_amd/build.py``).

bf16 tensors are ``torch.bfloat16``; FP8 codes are ``torch.uint8`` holding
OCP E4M3 (or E4M3FNUZ) bit patterns; int8 codes are ``torch.int8``; int4
codes are ``torch.uint8`` [N, K/2] (low nibble = even k, value c + 8).
"""

from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlin.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libqlin.so not found at {LIB_PATH}: build it with "
        "`python quantized_linear_layers_amd/build.py` (hipcc, gfx950)")

_lib = C.CDLL(LIB_PATH)

# ---------------------------------------------------------------- constants
OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_UNSUPPORTED, ERR_HIP = range(7)
E4M3, E4M3FNUZ, INT8 = 0, 1, 2
OUT_BF16, OUT_F32 = 0, 1
KV_BF16, KV_E4M3 = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_RAMP = range(4)
OP_GEMM_FP8, OP_GEMM_W8A8, OP_GEMM_W4A16, OP_LINEAR_FP8, OP_LINEAR_W8A8 = range(5)

_P, _I64, _INT, _SZ, _F32, _F64 = C.c_void_p, C.c_int64, C.c_int, C.c_size_t, C.c_float, C.c_double


class _KVCache(C.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("pages", _I64),
                ("kv_heads", _I64), ("page_size", _I64), ("head_dim", _I64), ("fmt", _INT)]


class _KVBatch(C.Structure):
    _fields_ = [("q_start", _P), ("kv_len", _P), ("page_table", _P), ("batch", _I64),
                ("table_cols", _I64), ("max_q", _I64)]


class _RopePlan(C.Structure):
    _fields_ = [("turns", _P), ("rot", _I64), ("interleaved", _INT), ("magnitude", _F32)]


class _KVPool(C.Structure):
    _fields_ = [("free_pages", _P), ("count", _P), ("pages", _I64), ("page_size", _I64)]


class _KVTables(C.Structure):
    _fields_ = [("page_table", _P), ("q_start", _P), ("kv_len", _P), ("slots", _P), ("positions", _P),
                ("batch", _I64), ("table_cols", _I64)]


class _Tree(C.Structure):
    _fields_ = [("mask", _P), ("positions", _P), ("words", _I64)]


class _HeadNorm(C.Structure):
    _fields_ = [("q_weight", _P), ("k_weight", _P), ("v_weight", _P), ("eps", _F32), ("offset", _F32),
                ("values", _INT)]


_SIGS = {
    "qlin_abi_version": (_INT, []),
    "qlin_status_str": (C.c_char_p, [_INT]),
    "qlin_last_hip_error": (_INT, []),
    "qlin_repack_q4_0": (_INT, [_P, _I64, _I64, _P, _P, _P, _P]),
    "qlin_repack_fp8": (_INT, [_P, _P, _I64, _I64, _INT, _P, _P, _P]),
    "qlin_repack_int8": (_INT, [_P, _P, _I64, _I64, _P, _P, _P]),
    "qlin_fp8_fnuz_to_ocp": (_INT, [_P, _P, _I64, _I64, _P, _P, _P, _P]),
    "qlin_dequant_q4_bf16": (_INT, [_P, _P, _I64, _I64, _P, _P]),
    "qlin_quant_act": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _P, _P]),
    "qlin_quant_weight": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P]),
    "qlin_embed_q4": (_INT, [_P, _I64, _P, _P, _I64, _I64, _P, _P]),
    "qlin_fp8_encode_f32": (_INT, [_P, _I64, _INT, _P, _P]),
    "qlin_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64]),
    "qlin_workspace_init": (_INT, [_P, _SZ, _P]),
    "qlin_gemm_fp8": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _INT, _P, _SZ, _P]),
    "qlin_gemm_w8a8": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _INT, _P, _SZ, _P]),
    "qlin_gemm_w4a16": (_INT, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _INT, _P, _SZ, _P]),
    "qlin_linear_fp8": (_INT, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "qlin_linear_w8a8": (_INT, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "qlin_moe_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _INT]),
    "qlin_moe_workspace_layout": (_INT, [_I64, _I64, _I64, _I64, _INT, C.POINTER(_SZ)]),
    "qlin_moe_fp8": (_INT, [_P, _I64, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _P, _P, _P,
                            _SZ, _P]),
    "qlin_moe_fp8_noalloc": (_INT, [_P, _I64, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _P, _P,
                                    _P]),
    "qlin_moe_fp8_swiglu_oai": (_INT, [_P, _I64, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _P,
                                       C.c_float, C.c_float, C.c_float, _P, _P, _SZ, _P]),
    "qlin_moe_w4a16_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _INT]),
    "qlin_moe_w4a16_workspace_layout": (_INT, [_I64, _I64, _I64, _I64, _INT, C.POINTER(_SZ)]),
    "qlin_moe_w4a16": (_INT, [_P, _I64, _I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _P, _P, _P,
                              _SZ, _P]),
    "qlin_rope_turns": (_INT, [_I64, _F64, _INT, _F64, _F64, _F64, _F64, C.POINTER(_F64)]),
    "qlin_rope": (_INT, [_P, _I64, _I64, _I64, _I64, _P, C.POINTER(_RopePlan), _INT, _P, _I64, _P]),
    "qlin_kv_append": (_INT, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _P, _I64, _P, _I64,
                              C.POINTER(_RopePlan), _P, _P, _I64, _I64, _P, _I64, _P]),
    "qlin_kv_append_norm": (_INT, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _P, _I64, _P, _I64,
                                   C.POINTER(_HeadNorm), C.POINTER(_RopePlan), _P, _P, _I64, _I64, _P, _I64, _P]),
    "qlin_norm_rope": (_INT, [_P, _I64, _I64, _I64, _I64, C.POINTER(_HeadNorm), _P, C.POINTER(_RopePlan), _P, _I64,
                              _P]),
    "qlin_attn_workspace_bytes": (_SZ, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _I64]),
    "qlin_attn_paged": (_INT, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _P, _I64, _I64, _F32,
                               _INT, _I64, _P, _I64, _P, _P, _SZ, _P]),
    "qlin_attn_tree": (_INT, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _P, _I64, _I64, _F32,
                              C.POINTER(_Tree), _I64, _P, _I64, _P, _P, _SZ, _P]),
    "qlin_kv_reserve": (_INT, [C.POINTER(_KVPool), C.POINTER(_KVTables), _I64, _P, _P, _P]),
    "qlin_kv_release": (_INT, [C.POINTER(_KVPool), C.POINTER(_KVTables), _P, _P]),
    "qlin_kv_keep": (_INT, [C.POINTER(_KVCache), _I64, C.POINTER(_KVBatch), _P, _I64, _P, _P, _P]),
    "qlin_attn_tree_workspace_bytes": (_SZ, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _I64]),
    "qlin_attn_tree_plan": (_INT, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _I64, _I64, C.POINTER(_I64)]),
    "qlin_tree_plan": (_INT, [C.POINTER(_KVBatch), _I64, _P, _I64, _P, _P, _P]),
    "qlin_attn_plan": (_INT, [C.POINTER(_KVCache), C.POINTER(_KVBatch), _I64, _I64, _I64, C.POINTER(_I64)]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class QlinError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.qlin_status_str(status).decode()
        if status == ERR_HIP:
            msg += f" (hipError {_lib.qlin_last_hip_error()})"
        super().__init__(f"{fn}: {msg}")
        self.status = status


def lib():
    """The raw ctypes handle of libqlin.so."""
    return _lib


def _call(name: str, *args):
    st = getattr(_lib, name)(*args)
    if st != OK:
        raise QlinError(name, st)


def _ptr(t: torch.Tensor | None):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return C.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_FMT = {"e4m3": E4M3, "e4m3fnuz": E4M3FNUZ, "int8": INT8, E4M3: E4M3, E4M3FNUZ: E4M3FNUZ,
        INT8: INT8}

# ---------------------------------------------------------------- workspace
# Buffers are cached per (device, stream): calls on one stream are ordered,
# so they may share a buffer, while calls on two streams may overlap and
# must not share split-K counters, partial sums or MoE stage data. A buffer
# that a call outgrows is replaced by one at least twice its size, and the
# old one is kept alive until the process ends: a HIP graph captured
# earlier, or a kernel still queued on the stream, may hold its address.
# (The retired buffers add up to less than the live one.)
_ws_cache: dict[tuple[int, int], torch.Tensor] = {}
_scratch_cache: dict[tuple[int, int], torch.Tensor] = {}
_retired: list[torch.Tensor] = []


def _cache_key(device: torch.device) -> tuple[int, int]:
    idx = device.index if device.index is not None else torch.cuda.current_device()
    return idx, torch.cuda.current_stream(idx).cuda_stream


def _cached(cache, nbytes: int, device: torch.device, zero: bool) -> torch.Tensor:
    key = _cache_key(device)
    ws = cache.get(key)
    if ws is None or ws.numel() < nbytes:
        size = max(nbytes, 1 << 20, 0 if ws is None else 2 * ws.numel())
        new = (torch.zeros if zero else torch.empty)(size, dtype=torch.uint8,
                                                     device=torch.device("cuda", key[0]))
        if ws is not None:
            _retired.append(ws)
        cache[key] = ws = new
    return ws


def workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    """Zero-initialised workspace of at least nbytes for the current stream
    of `device` (kept for reuse; the library leaves its counter area zero
    after every call)."""
    return _cached(_ws_cache, nbytes, device, True)


def scratch(nbytes: int, device: torch.device) -> torch.Tensor:
    """Scratch of at least nbytes for the current stream of `device`, for
    calls that overwrite their whole workspace (the MoE blocks). Kept apart
    from `workspace`, whose counter area the split-K GEMMs need to find
    zero."""
    return _cached(_scratch_cache, nbytes, device, False)


def workspace_bytes(op: int, M: int, N: int, K: int) -> int:
    return int(_lib.qlin_workspace_bytes(op, M, N, K))


# ---------------------------------------------------------------- repacks
def repack_q4_0(w: torch.Tensor):
    """bf16 QAT weight [N,K] -> (codes u8 [N,K/2], steps bf16 [N,K/32],
    n_ambiguous int64 [1] on device)."""
    _check(w, "w", torch.bfloat16, 2)
    N, K = w.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    steps = torch.empty((N, K // 32), dtype=torch.bfloat16, device=w.device)
    amb = torch.empty(1, dtype=torch.int64, device=w.device)
    _call("qlin_repack_q4_0", _ptr(w), N, K, _ptr(codes), _ptr(steps), _ptr(amb), _stream(w.device))
    return codes, steps, amb


def repack_fp8(codes: torch.Tensor, steps: torch.Tensor, fmt="e4m3"):
    """q4 grid -> (FP8 codes u8 [N,K], per-channel scale f32 [N])."""
    _check(codes, "codes", torch.uint8, 2)
    _check(steps, "steps", torch.bfloat16, 2)
    N, K = codes.shape[0], codes.shape[1] * 2
    wq = torch.empty((N, K), dtype=torch.uint8, device=codes.device)
    ws = torch.empty(N, dtype=torch.float32, device=codes.device)
    _call("qlin_repack_fp8", _ptr(codes), _ptr(steps), N, K, _FMT[fmt], _ptr(wq), _ptr(ws),
          _stream(codes.device))
    return wq, ws


def repack_int8(codes: torch.Tensor, steps: torch.Tensor):
    _check(codes, "codes", torch.uint8, 2)
    _check(steps, "steps", torch.bfloat16, 2)
    N, K = codes.shape[0], codes.shape[1] * 2
    wq = torch.empty((N, K), dtype=torch.int8, device=codes.device)
    ws = torch.empty(N, dtype=torch.float32, device=codes.device)
    _call("qlin_repack_int8", _ptr(codes), _ptr(steps), N, K, _ptr(wq), _ptr(ws),
          _stream(codes.device))
    return wq, ws


def fp8_fnuz_to_ocp(w_fnuz: torch.Tensor, s_in: torch.Tensor):
    """E4M3FNUZ weights + scales -> (OCP codes, scales, n_inexact int64 [1])."""
    _check(w_fnuz, "w_fnuz", torch.uint8, 2)
    _check(s_in, "s_in", torch.float32, 1)
    N, K = w_fnuz.shape
    wo = torch.empty_like(w_fnuz)
    so = torch.empty_like(s_in)
    bad = torch.empty(1, dtype=torch.int64, device=w_fnuz.device)
    _call("qlin_fp8_fnuz_to_ocp", _ptr(w_fnuz), _ptr(s_in), N, K, _ptr(wo), _ptr(so), _ptr(bad),
          _stream(w_fnuz.device))
    return wo, so, bad


def dequant_q4_bf16(codes: torch.Tensor, steps: torch.Tensor) -> torch.Tensor:
    _check(codes, "codes", torch.uint8, 2)
    _check(steps, "steps", torch.bfloat16, 2)
    N, K = codes.shape[0], codes.shape[1] * 2
    out = torch.empty((N, K), dtype=torch.bfloat16, device=codes.device)
    _call("qlin_dequant_q4_bf16", _ptr(codes), _ptr(steps), N, K, _ptr(out), _stream(codes.device))
    return out


# ---------------------------------------------------------------- quantisers
def quant_act(a: torch.Tensor, fmt="e4m3", out=None):
    """bf16 [M,K] (row stride may exceed K) -> (codes [M,K], scale f32 [M]).
    `out` may pass preallocated (codes, scale) tensors."""
    if not (isinstance(a, torch.Tensor) and a.is_cuda and a.dtype == torch.bfloat16 and a.dim() == 2
            and a.stride(1) == 1):
        raise ValueError("a must be a 2-D bf16 device tensor with unit column stride")
    M, K = a.shape
    f = _FMT[fmt]
    if out is not None:
        q, s = out
        _check(q, "out codes", torch.int8 if f == INT8 else torch.uint8, 2)
        _check(s, "out scale", torch.float32, 1)
        if q.shape != (M, K) or s.numel() != M:
            raise ValueError("out shape mismatch")
    else:
        q = torch.empty((M, K), dtype=torch.int8 if f == INT8 else torch.uint8, device=a.device)
        s = torch.empty(M, dtype=torch.float32, device=a.device)
    _call("qlin_quant_act", _ptr(a), M, K, a.stride(0), f, _ptr(q), _ptr(s), _stream(a.device))
    return q, s


def fp8_encode_f32(x: torch.Tensor, fmt="e4m3") -> torch.Tensor:
    _check(x, "x", torch.float32)
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _call("qlin_fp8_encode_f32", _ptr(x), x.numel(), _FMT[fmt], _ptr(out), _stream(x.device))
    return out


# ---------------------------------------------------------------- GEMMs
def _out(M, N, dev, out_dtype):
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    return torch.empty((M, N), dtype=out_dtype, device=dev), (OUT_F32 if out_dtype == torch.float32
                                                              else OUT_BF16)


def gemm_fp8(a_q, a_scale, w_q, w_scale, out_dtype=torch.bfloat16, out=None):
    """Y = ((A_q . W_q^T) * a_scale[:,None]) * w_scale[None,:], OCP E4M3."""
    _check(a_q, "a_q", torch.uint8, 2)
    _check(w_q, "w_q", torch.uint8, 2)
    _check(a_scale, "a_scale", torch.float32, 1)
    _check(w_scale, "w_scale", torch.float32, 1)
    M, K = a_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K or a_scale.numel() != M or w_scale.numel() != N:
        raise ValueError("shape mismatch")
    y, od = (out, OUT_F32 if out.dtype == torch.float32 else OUT_BF16) if out is not None else \
        _out(M, N, a_q.device, out_dtype)
    nb = workspace_bytes(OP_GEMM_FP8, M, N, K)
    ws = workspace(nb, a_q.device)
    _call("qlin_gemm_fp8", _ptr(a_q), _ptr(a_scale), _ptr(w_q), _ptr(w_scale), M, N, K, _ptr(y), od,
          _ptr(ws), ws.numel(), _stream(a_q.device))
    return y


def gemm_w8a8(a_q, a_scale, w_q, w_scale, out_dtype=torch.bfloat16, out=None):
    """Y = ((float)(A_q . W_q^T) * a_scale) * w_scale, int32 accumulation."""
    _check(a_q, "a_q", torch.int8, 2)
    _check(w_q, "w_q", torch.int8, 2)
    _check(a_scale, "a_scale", torch.float32, 1)
    _check(w_scale, "w_scale", torch.float32, 1)
    M, K = a_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K or a_scale.numel() != M or w_scale.numel() != N:
        raise ValueError("shape mismatch")
    y, od = (out, OUT_F32 if out.dtype == torch.float32 else OUT_BF16) if out is not None else \
        _out(M, N, a_q.device, out_dtype)
    nb = workspace_bytes(OP_GEMM_W8A8, M, N, K)
    ws = workspace(nb, a_q.device)
    _call("qlin_gemm_w8a8", _ptr(a_q), _ptr(a_scale), _ptr(w_q), _ptr(w_scale), M, N, K, _ptr(y),
          od, _ptr(ws), ws.numel(), _stream(a_q.device))
    return y


def gemm_w4a16(a, codes, steps, out_dtype=torch.bfloat16, out=None):
    """Y = A . bf16(c * step)^T with group-32 int4 weights, bf16 activations."""
    if not (isinstance(a, torch.Tensor) and a.is_cuda and a.dtype == torch.bfloat16 and a.dim() == 2
            and a.stride(1) == 1):
        raise ValueError("a must be a 2-D bf16 device tensor with unit column stride")
    _check(codes, "codes", torch.uint8, 2)
    _check(steps, "steps", torch.bfloat16, 2)
    M, K = a.shape
    N = codes.shape[0]
    if codes.shape[1] * 2 != K or steps.shape != (N, K // 32):
        raise ValueError("shape mismatch")
    y, od = (out, OUT_F32 if out.dtype == torch.float32 else OUT_BF16) if out is not None else \
        _out(M, N, a.device, out_dtype)
    nb = workspace_bytes(OP_GEMM_W4A16, M, N, K)
    ws = workspace(nb, a.device)
    _call("qlin_gemm_w4a16", _ptr(a), a.stride(0), _ptr(codes), _ptr(steps), M, N, K, _ptr(y), od,
          _ptr(ws), ws.numel(), _stream(a.device))
    return y


def _linear(name, op, x, w_q, w_scale, wdtype, out=None):
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2
            and x.stride(1) == 1):
        raise ValueError("x must be a 2-D bf16 device tensor with unit column stride")
    _check(w_q, "w_q", wdtype, 2)
    _check(w_scale, "w_scale", torch.float32, 1)
    M, K = x.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K or w_scale.numel() != N:
        raise ValueError("shape mismatch")
    if out is not None:
        _check(out, "out", torch.bfloat16, 2)
        if out.shape != (M, N):
            raise ValueError("out shape mismatch")
        y = out
    else:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ws = workspace(workspace_bytes(op, M, N, K), x.device)
    _call(name, _ptr(x), x.stride(0), _ptr(w_q), _ptr(w_scale), M, N, K, _ptr(y), _ptr(ws),
          ws.numel(), _stream(x.device))
    return y


def linear_fp8(x, w_q, w_scale, out=None):
    """Per-token FP8 quantisation of x followed by the FP8 GEMM (bf16 out)."""
    return _linear("qlin_linear_fp8", OP_LINEAR_FP8, x, w_q, w_scale, torch.uint8, out)


def linear_w8a8(x, w_q, w_scale, out=None):
    """Per-token int8 quantisation of x followed by the int8 GEMM."""
    return _linear("qlin_linear_w8a8", OP_LINEAR_W8A8, x, w_q, w_scale, torch.int8, out)


# ---------------------------------------------------------------- MoE
def moe_workspace_layout(T, H, I, E, topk):
    offs = (C.c_size_t * 6)()
    _call("qlin_moe_workspace_layout", T, H, I, E, topk, offs)
    return [int(o) for o in offs]


def embed_q4(ids, codes, steps):
    """Rows ids [T] (int32) of an int4 table (codes u8 [V,D/2], steps bf16
    [V,D/32]) as bf16 [T,D]; ids outside [0,V) give zero rows."""
    _check(ids, "ids", torch.int32, 1)
    _check(codes, "codes", torch.uint8, 2)
    _check(steps, "steps", torch.bfloat16, 2)
    V, D2 = codes.shape
    D = 2 * D2
    if steps.shape != (V, D // 32):
        raise ValueError("shape mismatch")
    out = torch.empty((ids.numel(), D), dtype=torch.bfloat16, device=codes.device)
    _call("qlin_embed_q4", _ptr(ids), ids.numel(), _ptr(codes), _ptr(steps), V, D, _ptr(out),
          _stream(codes.device))
    return out


def quant_weight(w: torch.Tensor, fmt="e4m3"):
    """Online per-channel quantisation of a bf16 weight [N,K] (contiguous):
    (codes [N,K], scale f32 [N]), one scale per output channel."""
    _check(w, "w", torch.bfloat16, 2)
    N, K = w.shape
    f = _FMT[fmt]
    q = torch.empty((N, K), dtype=torch.int8 if f == INT8 else torch.uint8, device=w.device)
    s = torch.empty(N, dtype=torch.float32, device=w.device)
    _call("qlin_quant_weight", _ptr(w), N, K, f, _ptr(q), _ptr(s), _stream(w.device))
    return q, s


def moe_fp8(x, topk_ids, topk_w, w13, s13, w2, s2, return_stages=False, swiglu_oai=None):
    """FP8 MoE block. x [T,H] bf16; topk_ids int32 [T,k]; topk_w f32 [T,k];
    w13 u8 [E,2I,H], s13 f32 [E,2I]; w2 u8 [E,H,I], s2 f32 [E,H].
    swiglu_oai: None for SiLU(g)*u, or (alpha, beta, limit) for SwiGLU-OAI."""
    _check(x, "x", torch.bfloat16, 2)
    _check(topk_ids, "topk_ids", torch.int32, 2)
    _check(topk_w, "topk_w", torch.float32, 2)
    _check(w13, "w13", torch.uint8, 3)
    _check(s13, "s13", torch.float32, 2)
    _check(w2, "w2", torch.uint8, 3)
    _check(s2, "s2", torch.float32, 2)
    T, H = x.shape
    E, I2, H2 = w13.shape
    I = I2 // 2
    topk = topk_ids.shape[1]
    if H2 != H or w2.shape != (E, H, I) or s13.shape != (E, I2) or s2.shape != (E, H) or \
            topk_w.shape != topk_ids.shape or topk_ids.shape[0] != T:
        raise ValueError("shape mismatch")
    nb = int(_lib.qlin_moe_workspace_bytes(T, H, I, E, topk))
    ws = scratch(nb, x.device) if not return_stages else \
        torch.empty(max(nb, 256), dtype=torch.uint8, device=x.device)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if swiglu_oai is None:
        _call("qlin_moe_fp8", _ptr(x), T, H, I, E, topk, _ptr(topk_ids), _ptr(topk_w), _ptr(w13),
              _ptr(s13), _ptr(w2), _ptr(s2), _ptr(y), _ptr(ws), ws.numel(), _stream(x.device))
    else:
        alpha, beta, limit = (float(v) for v in swiglu_oai)
        _call("qlin_moe_fp8_swiglu_oai", _ptr(x), T, H, I, E, topk, _ptr(topk_ids), _ptr(topk_w),
              _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), alpha, beta, limit, _ptr(y), _ptr(ws),
              ws.numel(), _stream(x.device))
    if not return_stages:
        return y
    o = moe_workspace_layout(T, H, I, E, topk)
    R = T * topk

    def view(off, n, dt):
        return ws[off: off + n * torch.tensor([], dtype=dt).element_size()].view(dt)

    stages = dict(xq=view(o[0], T * H, torch.uint8).view(T, H), sx=view(o[1], T, torch.float32),
                  act=view(o[2], R * I, torch.float32).view(R, I),
                  aq=view(o[3], R * I, torch.uint8).view(R, I), sa=view(o[4], R, torch.float32),
                  d=view(o[5], R * H, torch.float32).view(R, H))
    return y, stages


MOE_NOALLOC_MAX_BYTES = 64 << 20


def moe_fp8_noalloc(x, topk_ids, topk_w, w13, s13, w2, s2, out=None):
    """The FP8 MoE block through the allocation-free entry point: stage
    buffers in the library's static per-GPU array (calls that overlap on one
    GPU race). `out` may pass a preallocated y [T,H] bf16."""
    _check(x, "x", torch.bfloat16, 2)
    _check(topk_ids, "topk_ids", torch.int32, 2)
    _check(topk_w, "topk_w", torch.float32, 2)
    _check(w13, "w13", torch.uint8, 3)
    _check(s13, "s13", torch.float32, 2)
    _check(w2, "w2", torch.uint8, 3)
    _check(s2, "s2", torch.float32, 2)
    T, H = x.shape
    E, I2, H2 = w13.shape
    I = I2 // 2
    topk = topk_ids.shape[1]
    if H2 != H or w2.shape != (E, H, I) or s13.shape != (E, I2) or s2.shape != (E, H) or \
            topk_w.shape != topk_ids.shape or topk_ids.shape[0] != T:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    else:
        _check(out, "out", torch.bfloat16, 2)
        if out.shape != (T, H):
            raise ValueError("out shape mismatch")
    _call("qlin_moe_fp8_noalloc", _ptr(x), T, H, I, E, topk, _ptr(topk_ids), _ptr(topk_w), _ptr(w13),
          _ptr(s13), _ptr(w2), _ptr(s2), _ptr(out), _stream(x.device))
    return out


def moe_w4a16(x, topk_ids, topk_w, codes13, steps13, codes2, steps2, return_stages=False):
    """W4A16 MoE block. x [T,H] bf16; topk_ids int32 [T,k]; topk_w f32 [T,k];
    codes13 u8 [E,2I,H/2], steps13 bf16 [E,2I,H/32]; codes2 u8 [E,H,I/2],
    steps2 bf16 [E,H,I/32]."""
    _check(x, "x", torch.bfloat16, 2)
    _check(topk_ids, "topk_ids", torch.int32, 2)
    _check(topk_w, "topk_w", torch.float32, 2)
    _check(codes13, "codes13", torch.uint8, 3)
    _check(steps13, "steps13", torch.bfloat16, 3)
    _check(codes2, "codes2", torch.uint8, 3)
    _check(steps2, "steps2", torch.bfloat16, 3)
    T, H = x.shape
    E, I2, H2 = codes13.shape
    I = I2 // 2
    topk = topk_ids.shape[1]
    if H2 * 2 != H or codes2.shape != (E, H, I // 2) or steps13.shape != (E, I2, H // 32) or \
            steps2.shape != (E, H, I // 32) or topk_w.shape != topk_ids.shape or topk_ids.shape[0] != T:
        raise ValueError("shape mismatch")
    nb = int(_lib.qlin_moe_w4a16_workspace_bytes(T, H, I, E, topk))
    ws = scratch(nb, x.device) if not return_stages else \
        torch.empty(max(nb, 256), dtype=torch.uint8, device=x.device)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _call("qlin_moe_w4a16", _ptr(x), T, H, I, E, topk, _ptr(topk_ids), _ptr(topk_w), _ptr(codes13),
          _ptr(steps13), _ptr(codes2), _ptr(steps2), _ptr(y), _ptr(ws), ws.numel(), _stream(x.device))
    if not return_stages:
        return y
    offs = (_SZ * 2)()
    _call("qlin_moe_w4a16_workspace_layout", T, H, I, E, topk, offs)
    R = T * topk
    act = ws[offs[0]: offs[0] + R * I * 2].view(torch.bfloat16).view(R, I)
    d = ws[offs[1]: offs[1] + R * H * 4].view(torch.float32).view(R, H)
    return y, dict(act=act, d=d)


# ---------------------------------------------------------------- attention
# torch's own raw queries, where it has them: a Stream object costs more host time than a
# small launch, and the device's number a quarter of a microsecond
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _rows_arg(t, name, dev, head_dim, heads=None):
    """(rows, heads, row stride) of a bf16 tensor [T, heads, head_dim] on `dev` whose
    heads lie together; its rows may be further apart (a slice of a fused QKV
    projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}, got {t.device}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must have 3 dims, got {tuple(shape)}")
    T, H, D = shape
    if D != head_dim or (heads is not None and H != heads):
        raise ValueError(f"{name}: expected {'any' if heads is None else heads} heads of {head_dim}, got {H} of {D}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and H > 1):
        raise ValueError(f"{name}: the heads of a row must lie together")
    return T, H, s0 if T > 1 else H * D  # (the stride of a single row says nothing)


def _like(t):
    """A new contiguous tensor of t's shape."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _int64(x, name):
    """x as an int that ctypes hands over whole (beyond 64 bits it would wrap)."""
    x = int(x)
    if not -1 << 63 <= x < 1 << 63:
        raise ValueError(f"{name} must fit 64 bits, got {x}")
    return x


def _positions_arg(t, dev, T):
    _check(t, "positions", torch.int32, 1)
    if t.device != dev or t.numel() != T:
        raise ValueError(f"positions must be [T] on {dev}")
    return t.data_ptr()


def _on(dev, want, name):
    if dev != want:
        raise ValueError(f"{name} is on {dev}, expected {want}")


def _enqueue(dev: torch.device, fn, *args):
    """A library call on the current stream of `dev`, the current device."""
    st = fn(*args, _raw_stream(dev.index))
    if st != OK:
        raise QlinError(fn.__name__, st)


# An attention workspace beyond this is not kept between calls.
_ATTN_WS_KEEP = 64 << 20


def _attn_workspace(nbytes: int, dev: torch.device):
    """A workspace whose counter area is zero: the stream's own (`workspace`), or
    one of its own for a call that is being captured (two graphs of one stream
    may be replayed at once) and for a very large one."""
    if nbytes <= _ATTN_WS_KEEP and not torch.cuda.is_current_stream_capturing():
        ws = _ws_cache.get((dev.index, _raw_stream(dev.index)))
        return ws if ws is not None and ws.numel() >= nbytes else workspace(nbytes, dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws[:65536].zero_()
    return ws


class Rope:
    """A rotary plan: the frequencies (fp64, on `device`) of `rot_dim` turning
    values of a head of `head_dim` (default: all), and the pairs' layout: (i, i +
    rot_dim/2), or (2i, 2i + 1) if `interleaved`. `scaling` is None, ("linear",
    factor), ("base", factor) or ("ramp", factor, trained_len, low, high): see
    qlin_rope_turns. `magnitude` scales the rotated values (YaRN: 0.1 ln(factor)
    + 1 with ("ramp", factor, trained_len, 1, 32)). The ramp blends linearly in
    the number of turns, as YaRN's text defines it; model code that blends
    linearly in the pair's index gives other frequencies: take such a
    checkpoint's own by `turns` [rot_dim / 2] (tensor or sequence of floats: turns
    a position, inv_freq / 2 pi), which replaces base and scaling."""

    _RULES = {"linear": (ROPE_LINEAR, 1), "base": (ROPE_BASE, 1), "ramp": (ROPE_RAMP, 4)}

    def __init__(self, head_dim: int, rot_dim: int | None = None, base: float = 10000.0,
                 interleaved: bool = False, scaling=None, magnitude: float = 1.0, device="cuda", turns=None):
        self.head_dim, self.rot_dim = int(head_dim), int(head_dim if rot_dim is None else rot_dim)
        self.interleaved, self.magnitude = bool(interleaved), float(magnitude)
        if self.rot_dim > self.head_dim:
            raise ValueError("rot_dim must not exceed head_dim")
        rule, args = ROPE_PLAIN, []
        if scaling is not None:
            if turns is not None:
                raise ValueError("turns replaces the frequency rule: no scaling with it")
            if scaling[0] not in self._RULES or len(scaling) - 1 != self._RULES[scaling[0]][1]:
                raise ValueError(f"scaling {scaling!r}: expected one of {sorted(self._RULES)} and its arguments")
            rule, args = self._RULES[scaling[0]][0], [float(x) for x in scaling[1:]]
        args += [1.0, 1.0, 0.0, 1.0][len(args):]
        out = (_F64 * max(self.rot_dim // 2, 1))()
        _call("qlin_rope_turns", self.rot_dim, float(base), rule, *args, out)
        if turns is not None:
            given = torch.as_tensor(turns, dtype=torch.float64)
            if tuple(given.shape) != (self.rot_dim // 2,) or not bool(torch.isfinite(given).all()):
                raise ValueError("turns must be rot_dim / 2 finite values")
            out = given.tolist()
        self.turns = torch.tensor(list(out), dtype=torch.float64, device=device)
        if not self.turns.is_cuda:
            raise ValueError("device must be a GPU")
        self.device = self.turns.device
        self._c = _RopePlan(self.turns.data_ptr(), self.rot_dim, int(self.interleaved), self.magnitude)
        self._ref = C.byref(self._c)


class HeadNorm:
    """Norms of single heads: x / sqrt(mean(x^2) + eps) * (offset + weight), weights
    bf16 [D] on the GPU, or None for a part without one. Queries and keys are
    normalised, values if `values` or if they have a weight. offset=1.0 for weights
    that are stored less one. Without any weight, head_dim and device are taken from
    the arguments."""

    def __init__(self, q_weight=None, k_weight=None, v_weight=None, eps: float = 1e-6, offset: float = 0.0,
                 values=None, head_dim: int | None = None, device="cuda"):
        if values is not None and not values and v_weight is not None:
            raise ValueError("v_weight without values")
        self.values = v_weight is not None if values is None else bool(values)
        self.weights = {"q_weight": q_weight, "k_weight": k_weight, "v_weight": v_weight}
        self.eps, self.offset = float(eps), float(offset)
        self.head_dim = None if head_dim is None else int(head_dim)
        self.device = None
        for name, w in self.weights.items():
            if w is None:
                continue
            _check(w, name, torch.bfloat16, 1)
            if self.head_dim is None:
                self.head_dim = w.numel()
            if w.numel() != self.head_dim:
                raise ValueError(f"{name} must be [{self.head_dim}]")
            if self.device is None:
                self.device = w.device
            _on(w.device, self.device, name)
        if self.head_dim is None:
            raise ValueError("head_dim is needed without weights")
        if self.device is None:
            self.device = torch.empty(0, device=device).device
        if self.device.type != "cuda":
            raise ValueError("device must be a GPU")
        self._c = _HeadNorm(*(None if w is None else w.data_ptr() for w in self.weights.values()), self.eps,
                            self.offset, int(self.values))
        self._ref = C.byref(self._c)


class PagedKV:
    """A paged key/value cache: k, v [pages, kv_heads, page_size, head_dim], bf16,
    or uint8 E4M3 codes with k_scale, v_scale f32 [pages, kv_heads, page_size].
    Wraps existing tensors; `PagedKV.empty` allocates them."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not isinstance(k, torch.Tensor) or k.dtype not in (torch.bfloat16, torch.uint8):
            raise TypeError("k must be a bfloat16 or uint8 tensor")
        _check(k, "k", k.dtype, 4)
        _check(v, "v", k.dtype, 4)
        if v.shape != k.shape:
            raise ValueError("k and v must have one shape")
        self.fmt = KV_BF16 if k.dtype == torch.bfloat16 else KV_E4M3
        if self.fmt == KV_E4M3:
            _check(k_scale, "k_scale", torch.float32, 3)
            _check(v_scale, "v_scale", torch.float32, 3)
            if k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3]:
                raise ValueError("scales must be [pages, kv_heads, page_size]")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        self.device = k.device
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _on(t.device, self.device, name)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        if self.head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        if self.page_size not in (16, 32, 64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256")

        def addr(t):
            return None if t is None else t.data_ptr()

        self._c = _KVCache(addr(k), addr(v), addr(k_scale), addr(v_scale), self.pages, self.kv_heads,
                           self.page_size, self.head_dim, self.fmt)
        self._ref = C.byref(self._c)

    @classmethod
    def empty(cls, pages, kv_heads, head_dim, page_size=64, fmt="bf16", device="cuda"):
        """An uninitialised cache; fmt "bf16" or "e4m3"."""
        if fmt not in ("bf16", "e4m3"):
            raise ValueError("fmt must be 'bf16' or 'e4m3'")
        shape = (pages, kv_heads, page_size, head_dim)
        dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
        t = [torch.empty(shape, dtype=dt, device=device) for _ in range(2)]
        if fmt == "e4m3":
            t += [torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*t)


class PagedLayers:
    """The caches of a model's layers, of one size and format, that share a page table:
    what `kv_keep` moves rows of in one call."""

    def __init__(self, caches):
        self.caches = tuple(caches)
        if not self.caches:
            raise ValueError("at least one cache")
        one = self.caches[0]
        for c in self.caches:
            _on(c.device, one.device, "cache")
            if c.k.shape != one.k.shape or c.fmt != one.fmt:
                raise ValueError("the caches must have one size and format")
        at = sorted((t.data_ptr(), t.numel() * t.element_size()) for c in self.caches
                    for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None and t.numel())
        if any(a + size > b for (a, size), (b, _) in zip(at, at[1:])):  # (rows would be moved twice)
            raise ValueError("the caches must not share memory")
        self.device = one.device
        self._c = (_KVCache * len(self.caches))(*(c._c for c in self.caches))


class PagedBatch:
    """New tokens of a batch of sequences: q_start int32 [B+1], kv_len int32 [B],
    page_table int32 [B, cols] (device tensors, read when a call runs) and
    max_q, at least the longest sequence's count of new tokens (its kernels are
    chosen by it). Contents as at qlin_kv_batch."""

    def __init__(self, q_start, kv_len, page_table, max_q: int):
        _check(q_start, "q_start", torch.int32, 1)
        _check(kv_len, "kv_len", torch.int32, 1)
        _check(page_table, "page_table", torch.int32, 2)
        B = kv_len.numel()
        if q_start.numel() != B + 1 or page_table.shape[0] != B:
            raise ValueError("q_start must be [B+1], kv_len [B] and page_table [B, cols]")
        self.device = q_start.device
        _on(kv_len.device, self.device, "kv_len")
        _on(page_table.device, self.device, "page_table")
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.max_q = _int64(max_q, "max_q")
        self.batch = B
        self._c = _KVBatch(q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), B,
                           page_table.shape[1], self.max_q)
        self._ref = C.byref(self._c)
        self._ws_bytes = {}


class PagePool:
    """The pages of a cache that no request has: free int32 [pages], of which the first
    count[0] are free, and count int32 [2] (count[1]: pages that the last reservation
    lacked). Wraps device tensors; `PagePool.full` makes a pool with all pages free."""

    def __init__(self, free, count, page_size: int):
        _check(free, "free", torch.int32, 1)
        _check(count, "count", torch.int32, 1)
        self.device = free.device
        _on(count.device, self.device, "count")
        if count.numel() != 2:
            raise ValueError("count must be [2]")
        self.page_size = int(page_size)
        if self.page_size not in (16, 32, 64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256")
        self.free, self.count, self.pages = free, count, free.numel()
        self._c = _KVPool(free.data_ptr(), count.data_ptr(), self.pages, self.page_size)
        self._ref = C.byref(self._c)

    @classmethod
    def full(cls, pages: int, page_size: int = 64, device="cuda"):
        """All `pages` free, the lowest taken first."""
        return cls(torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.tensor([pages, 0], dtype=torch.int32, device=device), page_size)


class PageTables:
    """The tables of a batch of requests over `pool`: page_table int32 [B, cols] (the
    requests' pages), and q_start, kv_len, slots and positions of at most max_tokens new
    tokens, max_q of one request, which `reserve` writes. `batch` is the PagedBatch of
    them. All of them stay in place, so a captured graph may hold the calls.

    max_q chooses kernels and bounds a tree (512 tokens, and a window): where one set of
    tables serves prompts and trees, the trees' steps take a batch of their own over the
    same tensors, PagedBatch(tables.q_start, tables.kv_len, tables.page_table, max_q). Tables
    of more than 4096 tokens are reserved in two launches, whatever the step's tokens."""

    def __init__(self, pool: PagePool, page_table, max_tokens: int, max_q: int):
        _check(page_table, "page_table", torch.int32, 2)
        dev = self.device = pool.device
        _on(page_table.device, dev, "page_table")
        B, cols = page_table.shape
        self.pool, self.page_table, self.max_tokens = pool, page_table, int(max_tokens)
        self.q_start = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.slots = torch.full((self.max_tokens,), -1, dtype=torch.int32, device=dev)
        self.positions = torch.zeros(self.max_tokens, dtype=torch.int32, device=dev)
        self.batch = PagedBatch(self.q_start, self.kv_len, page_table, max_q)
        self._c = _KVTables(page_table.data_ptr(), self.q_start.data_ptr(), self.kv_len.data_ptr(),
                            self.slots.data_ptr(), self.positions.data_ptr(), B, cols)
        self._ref = C.byref(self._c)

    def _lengths(self, t, name):
        _check(t, name, torch.int32, 1)
        if t.device != self.device or t.numel() != self._c.batch:
            raise ValueError(f"{name} must be [{self._c.batch}] on {self.device}")
        return t.data_ptr()

    def reserve(self, lengths, new_tokens) -> PagedBatch:
        """Room for new_tokens int32 [B] behind lengths int32 [B] cached tokens: pages
        from the pool into page_table, starts, lengths, slots and positions of the new
        tokens (qlin_kv_reserve). pool.count[1] tells what the pool lacked: if not 0, drop
        the step with release(lengths) before anything is kept. (Tokens behind the table's
        columns have no page either and are not counted there.)"""
        dev = self.device
        if dev.index != _current_device():
            with torch.cuda.device(dev):
                return self.reserve(lengths, new_tokens)
        _enqueue(dev, _lib.qlin_kv_reserve, self.pool._ref, self._ref, self.max_tokens,
                 self._lengths(lengths, "lengths"), self._lengths(new_tokens, "new_tokens"))
        return self.batch

    def release(self, lengths) -> None:
        """Pages behind each request's first lengths int32 [B] tokens, up to its kv_len,
        back to the pool (qlin_kv_release). Once after a `reserve` (of no new tokens, if
        requests end between steps): a second time would give back the same pages."""
        dev = self.device
        if dev.index != _current_device():
            with torch.cuda.device(dev):
                return self.release(lengths)
        _enqueue(dev, _lib.qlin_kv_release, self.pool._ref, self._ref, self._lengths(lengths, "lengths"))


class Tree:
    """Trees of a batch's new tokens: mask int64 [T, words] (bit u % 64 of word u / 64:
    the token sees its sequence's new token u) and positions int32 [T], or None (no
    window then). Contents as at qlin_tree; `Tree.empty` allocates them for
    `tree_plan`."""

    def __init__(self, mask, positions=None):
        _check(mask, "mask", torch.int64, 2)
        self.device, (self.tokens, self.words) = mask.device, mask.shape
        if positions is not None:
            _check(positions, "positions", torch.int32, 1)
            _on(positions.device, self.device, "positions")
            if positions.numel() != self.tokens:
                raise ValueError("mask must be [T, words] and positions [T]")
        self.mask, self.positions = mask, positions
        self._c = _Tree(mask.data_ptr(), None if positions is None else positions.data_ptr(), self.words)
        self._ref = C.byref(self._c)

    @classmethod
    def empty(cls, tokens: int, words: int = 1, device="cuda"):
        """Uninitialised masks of `words` * 64 new tokens a sequence, and positions."""
        return cls(torch.empty((tokens, words), dtype=torch.int64, device=device),
                   torch.empty((tokens,), dtype=torch.int32, device=device))


def tree_plan(batch: PagedBatch, parents, tree: Tree | None = None):
    """The masks and positions of a batch's trees from the tokens' parents int32 [T]
    (numbers among a sequence's new tokens, -1: it follows the tokens before): into
    `tree`, which is returned, or into a new one."""
    dev = batch.device
    _check(parents, "parents", torch.int32, 1)
    _on(parents.device, dev, "parents")
    T = parents.numel()
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return tree_plan(batch, parents, tree)
    if tree is None:
        tree = Tree.empty(T, max(1, -(-batch.max_q // 64)), dev)
    _on(tree.device, dev, "tree")
    if tree.tokens != T:
        raise ValueError("parents and tree differ in tokens")
    _enqueue(dev, _lib.qlin_tree_plan, batch._ref, T, parents.data_ptr(), tree.words, tree._c.mask,
             tree._c.positions)
    return tree


def rope(x, positions, plan: Rope, out=None, inverse=False):
    """Rotary positions of x [T, H, D] (bf16) at positions int32 [T] by
    `plan`; `out` may be x. inverse=True turns the other way (the gradient of the
    rotation)."""
    D, dev = plan.head_dim, plan.device
    T, H, ldx = _rows_arg(x, "x", dev, D)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return rope(x, positions, plan, out, inverse)
    pos = _positions_arg(positions, dev, T)
    if out is None:
        out, ldy = _like(x), H * D
    else:
        T2, _, ldy = _rows_arg(out, "out", dev, D, H)
        if T2 != T:
            raise ValueError("out shape mismatch")
    _enqueue(dev, _lib.qlin_rope, x.data_ptr(), ldx, T, H, D, pos, plan._ref, 1 if inverse else 0, out.data_ptr(), ldy)
    return out


def norm_rope(x, norm: HeadNorm, positions=None, plan: Rope | None = None, out=None):
    """Heads x [T, H, D] (bf16) normalised by `norm` (its q_weight), then turned by
    `plan` at positions int32 [T] if there is one: the queries of a layer that stores
    no keys. `out` may be x."""
    D, dev = norm.head_dim, norm.device
    T, H, ldx = _rows_arg(x, "x", dev, D)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return norm_rope(x, norm, positions, plan, out)
    if plan is not None:
        _on(plan.device, dev, "plan")
        if plan.head_dim != D:
            raise ValueError("plan and norm differ in head_dim")
        if positions is None:
            raise ValueError("a rotation needs positions")
    if out is None:
        out, ldy = _like(x), H * D
    else:
        T2, _, ldy = _rows_arg(out, "out", dev, D, H)
        if T2 != T:
            raise ValueError("out shape mismatch")
    _enqueue(dev, _lib.qlin_norm_rope, x.data_ptr(), ldx, T, H, D, norm._ref,
             None if positions is None else _positions_arg(positions, dev, T), None if plan is None else plan._ref,
             out.data_ptr(), ldy)
    return out


def kv_append(cache: PagedKV, batch: PagedBatch, k, v, rope: Rope | None = None, q=None, q_out=None,
              positions=None, norm: HeadNorm | None = None):
    """The new tokens' keys (turned by `rope`) and values [T, kv_heads, D] into the
    cache. With q [T, q_heads, D] also turns the queries: returned, or written to
    q_out (which may be q). positions int32 [T] replaces each token's place in
    its sequence as what the rotation uses. With `norm`, queries, keys (and values)
    are normalised head by head before."""
    D, dev = cache.head_dim, cache.device
    _on(batch.device, dev, "batch")
    T, _, ldk = _rows_arg(k, "k", dev, D, cache.kv_heads)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return kv_append(cache, batch, k, v, rope, q, q_out, positions, norm)
    T2, _, ldv = _rows_arg(v, "v", dev, D, cache.kv_heads)
    ldq = ldqo = heads = 0
    if q is not None:
        T3, heads, ldq = _rows_arg(q, "q", dev, D)
        if q_out is None:
            q_out, ldqo = _like(q), heads * D
        else:
            T4, _, ldqo = _rows_arg(q_out, "q_out", dev, D, heads)
            T3 = T3 if T4 == T3 else -1
    else:
        if q_out is not None:
            raise ValueError("q_out without q")
        T3 = T
    if T2 != T or T3 != T:
        raise ValueError("k, v, q and q_out must have the same number of rows")
    if rope is not None:
        _on(rope.device, dev, "rope")
        if rope.head_dim != D:
            raise ValueError("rope and cache differ in head_dim")
    args = (None if rope is None else rope._ref, None if positions is None else _positions_arg(positions, dev, T),
            None if q is None else q.data_ptr(), ldq, heads, None if q is None else q_out.data_ptr(), ldqo)
    if norm is None:
        _enqueue(dev, _lib.qlin_kv_append, cache._ref, batch._ref, T, k.data_ptr(), ldk, v.data_ptr(), ldv, *args)
    else:
        _on(norm.device, dev, "norm")
        if norm.head_dim != D:
            raise ValueError("norm and cache differ in head_dim")
        _enqueue(dev, _lib.qlin_kv_append_norm, cache._ref, batch._ref, T, k.data_ptr(), ldk, v.data_ptr(), ldv,
                 norm._ref, *args)
    return q_out


def kv_keep(layers: PagedLayers | PagedKV, batch: PagedBatch, path, kept, lengths=None):
    """After a step of drafted tokens: each sequence's accepted ones, path int32 [B, W]
    (numbers among its new tokens, ascending) of which the first kept int32 [B], become
    its first new tokens in every layer's cache. Returns the cached tokens that are left,
    int32 [B] (or writes them to `lengths`): what the next step starts from. Kept tokens
    count whether or not they had a page (PageTables.reserve)."""
    if isinstance(layers, PagedKV):
        layers = PagedLayers((layers,))
    dev, B = layers.device, batch.batch
    _on(batch.device, dev, "batch")
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return kv_keep(layers, batch, path, kept, lengths)
    _check(path, "path", torch.int32, 2)
    _check(kept, "kept", torch.int32, 1)
    if lengths is None:
        lengths = torch.empty_like(kept)
    _check(lengths, "lengths", torch.int32, 1)
    for name, t in (("path", path), ("kept", kept), ("lengths", lengths)):
        if t.device != dev or t.shape[0] != B:
            raise ValueError(f"{name} must have {B} rows on {dev}")
    _enqueue(dev, _lib.qlin_kv_keep, layers._c, len(layers.caches), batch._ref, path.data_ptr(), path.shape[1],
             kept.data_ptr(), lengths.data_ptr())
    return lengths


def attn_paged(cache: PagedKV, batch: PagedBatch, q, scale=None, causal=True, window=0, out=None,
               return_lse=False, tree: Tree | None = None):
    """Attention of the new tokens' queries q [T, q_heads, D] over the cache, which
    holds their keys already (kv_append): [T, q_heads, D] bf16, and with
    return_lse the rows' ln of the sum of exponentials, f32 [T, q_heads]. scale
    defaults to D ** -0.5; window > 0 limits each token to its last `window` keys.
    With `tree`, each new token sees the earlier ones of its sequence and those new
    ones that its mask names (qlin_attn_tree; a window is then at least max_q). Weights are
    rounded to bf16 before they multiply the values, sums and lse are f32. Rows
    of q outside every sequence are left as they are in `out` (undefined in a new
    one)."""
    D, dev = cache.head_dim, cache.device
    _on(batch.device, dev, "batch")
    T, heads, ldq = _rows_arg(q, "q", dev, D)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return attn_paged(cache, batch, q, scale, causal, window, out, return_lse, tree)
    if out is None:
        out, ldo = _like(q), heads * D
    else:
        T2, _, ldo = _rows_arg(out, "out", dev, D, heads)
        if T2 != T:
            raise ValueError("out shape mismatch")
    if tree is not None:
        _on(tree.device, dev, "tree")
        if tree.tokens != T:
            raise ValueError("q and tree differ in tokens")
        if not causal:
            raise ValueError("a tree's masks replace causal")
    lse = q.new_empty((T, heads), dtype=torch.float32) if return_lse else None
    # what the size depends on beside the batch's own
    key = (T, heads, D, cache.kv_heads, cache.page_size, cache.fmt, tree is None)
    nb = batch._ws_bytes.get(key)
    if nb is None:
        size = _lib.qlin_attn_workspace_bytes if tree is None else _lib.qlin_attn_tree_workspace_bytes
        nb = batch._ws_bytes[key] = size(cache._ref, batch._ref, T, heads)
    ws = _attn_workspace(nb, dev) if nb else None
    fn, mask = (_lib.qlin_attn_paged, 1 if causal else 0) if tree is None else (_lib.qlin_attn_tree, tree._ref)
    _enqueue(dev, fn, cache._ref, batch._ref, T, q.data_ptr(), ldq, heads,
             D ** -0.5 if scale is None else float(scale), mask, _int64(window, "window"),
             out.data_ptr(), ldo, None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), nb)
    return (out, lse) if return_lse else out
