"""Python binding of libtq, the B200 (sm_100a) TurboQuant KV-cache quantisation library.

Argument marshalling only: every function below checks tensor placement / dtype / contiguity,
passes raw device pointers and the current CUDA stream to the C ABI declared in include/tq.h,
and raises TQError on a non-zero status. All computation happens in libtq's CUDA kernels
(and, for tq_codebook_init, in its host C++). There is no fallback: if libtq.so is missing or a
tensor is not on a CUDA device, the call fails.

Names follow the C ABI. Tensors:
  x        [n, d]  float32 / bfloat16 (CUDA)
  codes    [n, d/32, b] int32 (bit planes, uint32 bit patterns)
  signs    [n, d/32] int32
  norms    [n] float16,  gammas [n] float16
  rot      uint8 buffer of tq_rotation_bytes(d) bytes (prepared by tq_rotation_prepare)
  table    [n_pos, rot_dim/2, 2] float32 (cos, sin) of tq_rope_table
  PagedKV  the packed cache in pages: the arrays above with leading axes [pages, Hkv, page_size]
  ws       uint8 workspace; a call that is given none takes one from the pool of the stream it launches on
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA = 0, 1, 2, 3
TQ_ERR_NOT_CONVERGED, TQ_ERR_DEVICE_TIMEOUT, TQ_ERR_WORKSPACE, TQ_ERR_DEVICE_INPUT = 4, 5, 6, 7
TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
TQ_ROPE_HALF, TQ_ROPE_PAIRS = 0, 1
TQ_ROPE_PLAIN, TQ_ROPE_LINEAR, TQ_ROPE_BLEND = 0, 1, 2


class TQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libtq status {status}: {message}")
        self.status = status


class Codebook(ctypes.Structure):
    """Mirror of tq_codebook (host POD)."""
    _fields_ = [
        ("d", ctypes.c_int32), ("bits", ctypes.c_int32), ("levels", ctypes.c_int32),
        ("iterations", ctypes.c_int32),
        ("c", ctypes.c_float * 16), ("t", ctypes.c_float * 16),
        ("c64", ctypes.c_double * 16), ("t64", ctypes.c_double * 16),
        ("distortion", ctypes.c_double),
    ]

    @property
    def centroids(self):
        return list(self.c)[: self.levels]

    @property
    def boundaries(self):
        return list(self.t)[: self.levels - 1]


class _PagedKV(ctypes.Structure):
    """Mirror of tq_paged_kv (host POD)."""
    _fields_ = [
        ("d", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("page_size", ctypes.c_int32), ("v_alg", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("k_codes", ctypes.c_void_p), ("k_norms", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("v_signs", ctypes.c_void_p), ("v_norms", ctypes.c_void_p), ("v_gammas", ctypes.c_void_p),
        ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32),
        ("ck", ctypes.c_float * 16), ("tk", ctypes.c_float * 16), ("cv", ctypes.c_float * 16), ("tv", ctypes.c_float * 16),
        ("k_half", ctypes.c_uint16 * 16), ("v_half", ctypes.c_uint16 * 16),
        ("k_unit", ctypes.c_float), ("v_unit", ctypes.c_float), ("ready", ctypes.c_uint32),
    ]


_lib = None

_P = ctypes.c_void_p
_I32, _I64, _SZ, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_CB = ctypes.POINTER(Codebook)
_KV = ctypes.POINTER(_PagedKV)
_D = ctypes.c_double

_SIGNATURES = {
    "tq_last_error": (ctypes.c_char_p, []),
    "tq_version": (ctypes.c_char_p, []),
    "tq_codebook_init": (_I32, [_I32, _I32, _CB]),
    "tq_rotation_bytes": (_SZ, [_I32]),
    "tq_rotation_prepare": (_I32, [_I32, _P, _P, _P, _SZ, _P]),
    "tq_encode_mse": (_I32, [_CB, _I64, _I32, _P, _I32, _P, _P, _P, _P]),
    "tq_encode_prod": (_I32, [_CB, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "tq_encode_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "tq_decode": (_I32, [_CB, _I64, _I32, _P, _P, _P, _P, _P, _P, _I32, _P]),
    "tq_encode_mse_mixed": (_I32, [_CB, _P, _I64, _I32, _P, _I32, _P, _P, _P, _P]),
    "tq_decode_mixed": (_I32, [_CB, _P, _I64, _I32, _P, _P, _P, _P, _I32, _P]),
    "tq_scores_workspace_bytes": (_SZ, [_I64, _I64, _I32, _I32]),
    "tq_scores": (_I32, [_CB, _I64, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "tq_attend_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I64, _I32]),
    "tq_attend_decode": (_I32, [_CB, _CB, _I32, _I32, _I32, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                _P, _F, _P, _P, _SZ, _P]),
    "tq_attend_decode_noalloc": (_I32, [_CB, _CB, _I32, _I32, _I32, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P,
                                        _P, _P, _P, _F, _P, _P]),
    "tq_attend_prefill_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I32, _I64, _I32]),
    "tq_attend_prefill": (_I32, [_CB, _CB, _I32, _I32, _I32, _I32, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P,
                                 _P, _P, _F, _P, _P, _SZ, _P]),
    "tq_attend_append_workspace_bytes": (_SZ, [_I32, _I32, _I32, _I64, _I32, _I32, _I32]),
    "tq_attend_append": (_I32, [_CB, _CB, _I32, _I32, _I32, _I64, _I64, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P,
                                _P, _P, _P, _P, _F, _P, _P, _SZ, _P]),
    "tq_rope_table": (_I32, [_I64, _I32, _D, _I32, _D, _D, _D, _D, _D, _P, _P]),
    "tq_rope": (_I32, [_I64, _I32, _I32, _I32, _I32, _I32, _P, _I64, _I64, _I32, _P, _P, _I64, _P, _I64, _I64, _P]),
    "tq_paged_kv_init": (_I32, [_CB, _CB, _I32, _I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _KV]),
    "tq_paged_append": (_I32, [_KV, _I64, _P, _I64, _P, _I64, _I32, _P, _P, _P, _I64, _I32, _I32, _P, _P]),
    "tq_paged_attend_workspace_bytes": (_SZ, [_KV, _I32, _I32, _I64, _I32, _I64]),
    "tq_paged_attend": (_I32, [_KV, _I32, _I32, _I64, _I32, _I64, _P, _I64, _I32, _P, _P, _P, _I32, _F, _F, _I32, _P,
                               _P, _P, _P, _P, _SZ, _P]),
    "tq_selftest_wait": (_I32, [ctypes.c_uint64, _P]),
    "tq_sync_check": (_I32, [_P]),
}


def lib() -> ctypes.CDLL:
    """The loaded libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtq.so not found at {LIB_PATH}; build it with "
                               "`python -m kv_cache_vector_encode_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name, None)
            if fn is None:
                continue
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != TQ_OK:
        raise TQError(status, lib().tq_last_error().decode())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _empty(shape, dtype, device, stream, keep=False):
    """torch.empty for a call that launches on `stream`: memory of that stream, so that what it waits for, and what may
    follow when it is released (a workspace when the call returns), is in that stream's order. keep: the tensor is the
    call's result, which the current stream may go on using until it is released."""
    import torch
    if stream is not None and device.type == "cuda":
        current = torch.cuda.current_stream(device)
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle != current.cuda_stream:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(handle, device=device)
            with torch.cuda.stream(stream):
                t = torch.empty(shape, dtype=dtype, device=device)
            if keep:
                t.record_stream(current)
            return t
    return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t, name, dtypes=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    return ctypes.c_void_p(t.data_ptr())


def _rotation(rot, d):
    """Address of a prepared rotation that is as large as one for d (the C calls take no size)."""
    import torch
    ptr = _ptr(rot, "rot", [torch.uint8])
    if rot.numel() < tq_rotation_bytes(d):
        raise ValueError(f"rot has {rot.numel()} bytes, a rotation prepared for d = {d} has {tq_rotation_bytes(d)}")
    return ptr


def _xdtype(t):
    import torch
    return {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}[t.dtype]


# ---- entry points ------------------------------------------------------------------------------

def tq_version() -> str:
    return lib().tq_version().decode()


def tq_codebook_init(d: int, bits: int) -> Codebook:
    cb = Codebook()
    _check(lib().tq_codebook_init(d, bits, ctypes.byref(cb)))
    return cb


@functools.lru_cache(maxsize=None)           # every call that takes a rotation asks for it
def tq_rotation_bytes(d: int) -> int:
    return int(lib().tq_rotation_bytes(d))


def tq_rotation_prepare(Pi, S, rot=None, stream=None):
    """Prepare the rotation buffer from device fp32 Pi, S (d x d); returns it."""
    import torch
    d = Pi.shape[0]
    if tuple(Pi.shape) != (d, d) or tuple(S.shape) != (d, d):
        raise ValueError("Pi and S must be [d, d]")
    nbytes = tq_rotation_bytes(d)
    if rot is None:
        rot = _empty(nbytes, torch.uint8, Pi.device, stream, keep=True)
    _check(lib().tq_rotation_prepare(d, _ptr(Pi, "Pi", [torch.float32]), _ptr(S, "S", [torch.float32]),
                                     _ptr(rot, "rot"), rot.numel(), _stream(stream)))
    return rot


def tq_encode_mse(cb: Codebook, x, rot, codes, norms, stream=None):
    import torch
    n, d = x.shape
    _check(lib().tq_encode_mse(ctypes.byref(cb), n, d, _ptr(x, "x", [torch.float32, torch.bfloat16]), _xdtype(x),
                               _rotation(rot, d), _ptr(codes, "codes", [torch.int32]),
                               _ptr(norms, "norms", [torch.float16]), _stream(stream)))


def tq_encode_workspace_bytes(n: int, d: int, alg: int) -> int:
    return int(lib().tq_encode_workspace_bytes(n, d, alg))


def tq_encode_prod(cb_bm1: Codebook, x, rot, codes, signs, norms, gammas, ws=None, stream=None):
    import torch
    n, d = x.shape
    wsb = tq_encode_workspace_bytes(n, d, 2)
    if ws is None and wsb > 0:
        ws = _empty(wsb, torch.uint8, x.device, stream)
    _check(lib().tq_encode_prod(ctypes.byref(cb_bm1), n, d, _ptr(x, "x", [torch.float32, torch.bfloat16]),
                                _xdtype(x), _rotation(rot, d), _ptr(codes, "codes", [torch.int32]),
                                _ptr(signs, "signs", [torch.int32]), _ptr(norms, "norms", [torch.float16]),
                                _ptr(gammas, "gammas", [torch.float16]), _ptr(ws, "ws", None, True),
                                ws.numel() if ws is not None else 0, _stream(stream)))


def tq_decode(cb: Codebook, rot, codes, norms, out, signs=None, gammas=None, stream=None):
    import torch
    n, d = out.shape
    _check(lib().tq_decode(ctypes.byref(cb), n, d, _rotation(rot, d), _ptr(codes, "codes", [torch.int32]),
                           _ptr(signs, "signs", [torch.int32], True), _ptr(norms, "norms", [torch.float16]),
                           _ptr(gammas, "gammas", [torch.float16], True),
                           _ptr(out, "out", [torch.float32, torch.bfloat16]), _xdtype(out), _stream(stream)))


_mixed_cache = {}


def _mixed_args(d: int, group_bits):
    """Host arrays of the mixed-width calls: the 4 codebooks of d (1..4 bits) and the group widths
    (made once per (d, widths); the codebooks come from the library's host solver)."""
    key = (int(d), tuple(int(x) for x in group_bits))
    if key not in _mixed_cache:
        G = d // 32
        if len(key[1]) != G:
            raise ValueError(f"group_bits needs {G} entries for d = {d}")
        cbs = (Codebook * 4)()
        for b in sorted(set(key[1])):
            if 1 <= b <= 4:
                cbs[b - 1] = tq_codebook_init(d, b)
        _mixed_cache[key] = (cbs, (ctypes.c_int32 * G)(*key[1]))
    return _mixed_cache[key]


def tq_encode_mse_mixed(group_bits, x, rot, codes, norms, stream=None):
    """Algorithm 1 with a width per group of 32 rotated coordinates; codes [n, sum(group_bits)] int32."""
    import torch
    n, d = x.shape
    cbs, gb = _mixed_args(d, group_bits)
    _check(lib().tq_encode_mse_mixed(cbs, gb, n, d, _ptr(x, "x", [torch.float32, torch.bfloat16]), _xdtype(x),
                                     _rotation(rot, d), _ptr(codes, "codes", [torch.int32]),
                                     _ptr(norms, "norms", [torch.float16]), _stream(stream)))


def tq_decode_mixed(group_bits, rot, codes, norms, out, stream=None):
    import torch
    n, d = out.shape
    cbs, gb = _mixed_args(d, group_bits)
    _check(lib().tq_decode_mixed(cbs, gb, n, d, _rotation(rot, d), _ptr(codes, "codes", [torch.int32]),
                                 _ptr(norms, "norms", [torch.float16]),
                                 _ptr(out, "out", [torch.float32, torch.bfloat16]), _xdtype(out), _stream(stream)))


def tq_scores_workspace_bytes(nq: int, n: int, d: int, k: int) -> int:
    return int(lib().tq_scores_workspace_bytes(nq, n, d, k))


def tq_scores(cb: Codebook, q, rot, codes, norms, signs=None, gammas=None, scores=None, k=0, topk_ids=None,
              topk_scores=None, ws=None, stream=None):
    import torch
    nq, d = q.shape
    n = norms.shape[0]
    wsb = tq_scores_workspace_bytes(nq, n, d, k)
    if ws is None:
        ws = _empty(max(wsb, 16), torch.uint8, q.device, stream)
    _check(lib().tq_scores(ctypes.byref(cb), nq, n, d, _ptr(q, "q", [torch.float32, torch.bfloat16]), _xdtype(q),
                           _rotation(rot, d), _ptr(codes, "codes", [torch.int32]),
                           _ptr(signs, "signs", [torch.int32], True), _ptr(norms, "norms", [torch.float16]),
                           _ptr(gammas, "gammas", [torch.float16], True),
                           _ptr(scores, "scores", [torch.float32], True), k,
                           _ptr(topk_ids, "topk_ids", [torch.int32], True),
                           _ptr(topk_scores, "topk_scores", [torch.float32], True),
                           _ptr(ws, "ws"), ws.numel(), _stream(stream)))


def tq_attend_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, d: int) -> int:
    return int(lib().tq_attend_workspace_bytes(B, Hq, Hkv, T, d))


def tq_attend_decode(cb_k: Codebook, cb_v: Codebook, q, rot, k_codes, k_norms, v_codes, v_norms, out,
                     v_signs=None, v_gammas=None, scale=None, ws=None, stream=None, k_signs=None, k_gammas=None):
    import torch
    B, Hq, d = q.shape
    Hkv, T = k_norms.shape[1], k_norms.shape[2]
    if scale is None:
        scale = 0.0                   # the library's default, 1/sqrt(d)
    wsb = tq_attend_workspace_bytes(B, Hq, Hkv, T, d)
    if ws is None:
        ws = _empty(max(wsb, 16), torch.uint8, q.device, stream)
    _check(lib().tq_attend_decode(ctypes.byref(cb_k), ctypes.byref(cb_v), B, Hq, Hkv, T, d,
                                  _ptr(q, "q", [torch.float32, torch.bfloat16]), _xdtype(q), _rotation(rot, d),
                                  _ptr(k_codes, "k_codes", [torch.int32]), _ptr(k_norms, "k_norms", [torch.float16]),
                                  _ptr(k_signs, "k_signs", [torch.int32], True),
                                  _ptr(k_gammas, "k_gammas", [torch.float16], True),
                                  _ptr(v_codes, "v_codes", [torch.int32]),
                                  _ptr(v_signs, "v_signs", [torch.int32], True),
                                  _ptr(v_norms, "v_norms", [torch.float16]),
                                  _ptr(v_gammas, "v_gammas", [torch.float16], True), float(scale),
                                  _ptr(out, "out", [torch.float32]), _ptr(ws, "ws"), ws.numel(), _stream(stream)))


def tq_attend_decode_noalloc(cb_k: Codebook, cb_v: Codebook, q, rot, k_codes, k_norms, v_codes, v_norms, out,
                             v_signs=None, v_gammas=None, scale=None, stream=None, k_signs=None, k_gammas=None):
    """tq_attend_decode with the library's fixed scratch array (no workspace, no allocation)."""
    import torch
    B, Hq, d = q.shape
    Hkv, T = k_norms.shape[1], k_norms.shape[2]
    if scale is None:
        scale = 0.0                   # the library's default, 1/sqrt(d)
    _check(lib().tq_attend_decode_noalloc(ctypes.byref(cb_k), ctypes.byref(cb_v), B, Hq, Hkv, T, d,
                                          _ptr(q, "q", [torch.float32, torch.bfloat16]), _xdtype(q), _rotation(rot, d),
                                          _ptr(k_codes, "k_codes", [torch.int32]),
                                          _ptr(k_norms, "k_norms", [torch.float16]),
                                          _ptr(k_signs, "k_signs", [torch.int32], True),
                                          _ptr(k_gammas, "k_gammas", [torch.float16], True),
                                          _ptr(v_codes, "v_codes", [torch.int32]),
                                          _ptr(v_signs, "v_signs", [torch.int32], True),
                                          _ptr(v_norms, "v_norms", [torch.float16]),
                                          _ptr(v_gammas, "v_gammas", [torch.float16], True), float(scale),
                                          _ptr(out, "out", [torch.float32]), _stream(stream)))


def tq_attend_prefill_workspace_bytes(B: int, Hq: int, Hkv: int, Qn: int, T: int, d: int) -> int:
    return int(lib().tq_attend_prefill_workspace_bytes(B, Hq, Hkv, Qn, T, d))


def tq_attend_prefill(cb_k: Codebook, cb_v: Codebook, q, rot, k_codes, k_norms, v_codes, v_norms, out,
                      v_signs=None, v_gammas=None, scale=None, ws=None, stream=None, k_signs=None, k_gammas=None):
    """Causal multi-query attention: q, out [B, Qn, Hq, d]; the cache [B][Hkv][T] holds the Qn new
    tokens in its last Qn slots (query j attends slots t <= T - Qn + j)."""
    import torch
    B, Qn, Hq, d = q.shape
    Hkv, T = k_norms.shape[1], k_norms.shape[2]
    if scale is None:
        scale = 0.0                   # the library's default, 1/sqrt(d)
    wsb = tq_attend_prefill_workspace_bytes(B, Hq, Hkv, Qn, T, d)
    if ws is None:
        ws = _empty(max(wsb, 16), torch.uint8, q.device, stream)
    _check(lib().tq_attend_prefill(ctypes.byref(cb_k), ctypes.byref(cb_v), B, Hq, Hkv, Qn, T, d,
                                   _ptr(q, "q", [torch.float32, torch.bfloat16]), _xdtype(q), _rotation(rot, d),
                                   _ptr(k_codes, "k_codes", [torch.int32]), _ptr(k_norms, "k_norms", [torch.float16]),
                                   _ptr(k_signs, "k_signs", [torch.int32], True),
                                   _ptr(k_gammas, "k_gammas", [torch.float16], True),
                                   _ptr(v_codes, "v_codes", [torch.int32]),
                                   _ptr(v_signs, "v_signs", [torch.int32], True),
                                   _ptr(v_norms, "v_norms", [torch.float16]),
                                   _ptr(v_gammas, "v_gammas", [torch.float16], True), float(scale),
                                   _ptr(out, "out", [torch.float32]), _ptr(ws, "ws"), ws.numel(), _stream(stream)))


TQ_ATTEND_NOALLOC_MAX_BYTES = 8 << 20


def tq_attend_append_workspace_bytes(B: int, Hq: int, Hkv: int, T_cur: int, d: int, k_bits: int,
                                     v_codebook_bits: int) -> int:
    return int(lib().tq_attend_append_workspace_bytes(B, Hq, Hkv, T_cur, d, k_bits, v_codebook_bits))


def tq_attend_append(cb_k: Codebook, cb_v: Codebook, q, rot, k_new, v_new, T_cur: int, k_codes, k_norms, v_codes,
                     v_signs, v_norms, v_gammas, out, scale=None, ws=None, stream=None):
    """Encode the new token's K / V of every slice into slot T_cur of the cache, then attend over slots
    [0, T_cur]. The cache tensors are [B][Hkv][T_max]... as for tq_attend_decode; k_new, v_new [B][Hkv][d]."""
    import torch
    B, Hq, d = q.shape
    Hkv, T_max = k_norms.shape[1], k_norms.shape[2]
    if k_new.dtype != v_new.dtype:
        raise TypeError("tq_attend_append: k_new and v_new must have the same dtype (one x_dtype for both)")
    if tuple(k_new.shape) != (B, Hkv, d) or tuple(v_new.shape) != (B, Hkv, d):
        raise ValueError(f"tq_attend_append: k_new / v_new must be [B, Hkv, d] = {(B, Hkv, d)}")
    if scale is None:
        scale = 0.0                   # the library's default, 1/sqrt(d)
    wsb = tq_attend_append_workspace_bytes(B, Hq, Hkv, T_cur, d, cb_k.bits, cb_v.bits)
    if ws is None:
        ws = _empty(max(wsb, 16), torch.uint8, q.device, stream)
    _check(lib().tq_attend_append(ctypes.byref(cb_k), ctypes.byref(cb_v), B, Hq, Hkv, T_cur, T_max, d,
                                  _ptr(q, "q", [torch.float32, torch.bfloat16]), _xdtype(q),
                                  _ptr(k_new, "k_new", [torch.float32, torch.bfloat16]),
                                  _ptr(v_new, "v_new", [torch.float32, torch.bfloat16]), _xdtype(k_new),
                                  _rotation(rot, d), _ptr(k_codes, "k_codes", [torch.int32]),
                                  _ptr(k_norms, "k_norms", [torch.float16]), _ptr(v_codes, "v_codes", [torch.int32]),
                                  _ptr(v_signs, "v_signs", [torch.int32]), _ptr(v_norms, "v_norms", [torch.float16]),
                                  _ptr(v_gammas, "v_gammas", [torch.float16]), float(scale),
                                  _ptr(out, "out", [torch.float32]), _ptr(ws, "ws"), ws.numel(), _stream(stream)))


# ---- rotary positions, packed cache in pages -----------------------------------------------------
# These are called once per layer and step, on few rows at a time, where the host's time is what a caller
# waits for: the checks below use the cheapest accessors (get_device() tells device and kind at once).

class _Torch:
    """What the checks need of torch, looked up once."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.f16 = torch.float32, torch.bfloat16, torch.float16
        self.i32, self.i64, self.u8 = torch.int32, torch.int64, torch.uint8
        self.code = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_stream = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)


_tc = None


def _torch() -> _Torch:
    global _tc
    if _tc is None:
        lib()
        _tc = _Torch()
    return _tc


def _current(t, name):
    """Index of the CUDA device that t is on, which has to be the current one (the calls launch there)."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device != _torch().current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return device


def _in(t, name, device, dtype, *shape):
    """Address of a contiguous tensor of this device, dtype and shape."""
    if t.get_device() != device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on device {device}")
    return t.data_ptr()


def _fits(*values, bits=32):
    """The integers that a caller gives have to fit their C types, which would cut them short."""
    most = 1 << (bits - 1)
    for v in values:
        if not -most <= v < most:
            raise ValueError(f"{v} does not fit {bits} bits")


def _table(table, device):
    """Address, positions and rotated dimensions of a tq_rope_table."""
    if table.get_device() != device or table.dtype is not _tc.f32 or table.dim() != 3 or not table.is_contiguous():
        raise ValueError(f"table must be a contiguous torch.float32 tensor [n_pos, rot_dim // 2, 2] on device {device}")
    n_pos, half, two = table.shape
    if two != 2:
        raise ValueError("table must be [n_pos, rot_dim // 2, 2]")
    return table.data_ptr(), n_pos, 2 * half


def _raw(stream, device):
    if stream is None:
        return _tc.raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def tq_rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, scaling: int = TQ_ROPE_PLAIN, factor: float = 1.0,
                  low_turns: float = 1.0, high_turns: float = 32.0, original_len: float = 0.0,
                  magnitude: float = 1.0, device="cuda", stream=None):
    """Table [n_pos, rot_dim // 2, 2] float32 of (cos, sin) for tq_rope and tq_paged_append."""
    import torch
    _fits(rot_dim, scaling)
    device = torch.device(device)
    table = _empty((n_pos, rot_dim // 2, 2), torch.float32, device, stream, keep=True)
    _current(table, "device")
    _check(lib().tq_rope_table(n_pos, rot_dim, base, scaling, factor, low_turns, high_turns, original_len, magnitude,
                               table.data_ptr(), _stream(stream)))
    return table


def tq_rope(x, positions, table, out=None, layout: int = TQ_ROPE_HALF, inverse: bool = False, stream=None):
    """Turns the heads of x [tokens, heads, d] (float32 / bfloat16 / float16, last axis contiguous) to positions
    [tokens] (int32; negative: a padding row, left as it is). out: x itself by default (in place).
    inverse=True turns the other way: the gradient with respect to x."""
    device = _current(x, "x")
    code = _tc.code.get(x.dtype)
    if code is None:
        raise ValueError(f"x: dtype {x.dtype} not float32 / bfloat16 / float16")
    tokens, heads, d = x.shape
    xt, xh, xd = os_ = x.stride()
    if out is None:
        out = x
    else:
        if out.shape != x.shape or out.dtype is not x.dtype or out.get_device() != device:
            raise ValueError("out must have the shape, dtype and device of x")
        os_ = out.stride()
    if xd != 1 or os_[2] != 1:
        raise ValueError("the last axis of x and out must be contiguous")
    pos = _in(positions, "positions", device, _tc.i32, tokens)
    tab, n_pos, rot_dim = _table(table, device)
    _fits(layout)
    status = _lib.tq_rope(tokens, heads, d, rot_dim, layout, 1 if inverse else 0, x.data_ptr(), xt, xh, code, pos, tab, n_pos,
                          out.data_ptr(), os_[0], os_[1], _raw(stream, device))
    if status:
        _check(status)
    return out


class PagedKV:
    """Handle of a packed cache in pages (tq_paged_kv): k_codes [pages, Hkv, page_size, d/32, b_k] int32,
    k_norms [pages, Hkv, page_size] float16, v_codes, v_norms likewise; v_signs [pages, Hkv, page_size, d/32]
    and v_gammas for values by Algorithm 2. It keeps the tensors alive."""

    def __init__(self, cb_k: Codebook, cb_v: Codebook, k_codes, k_norms, v_codes, v_norms, v_signs=None, v_gammas=None):
        self.device = device = _current(k_codes, "k_codes")
        if k_codes.dim() != 5:
            raise ValueError("k_codes must be [pages, Hkv, page_size, d/32, bits]")
        at, groups = tuple(k_codes.shape[:3]), k_codes.shape[3]
        if (v_signs is None) != (v_gammas is None):
            raise ValueError("v_signs and v_gammas go together")
        for name, t, shape in (("k_codes", k_codes, (*at, groups, cb_k.bits)), ("v_codes", v_codes, (*at, groups, cb_v.bits)),
                               ("k_norms", k_norms, at), ("v_norms", v_norms, at), ("v_signs", v_signs, (*at, groups)),
                               ("v_gammas", v_gammas, at)):
            if t is not None:
                _in(t, name, device, _tc.i32 if len(shape) > 3 else _tc.f16, *shape)
        self.tensors = (k_codes, k_norms, v_codes, v_norms, v_signs, v_gammas)
        self.num_pages, self.Hkv, self.page_size = at
        self.d = 32 * groups
        self.rot_bytes = tq_rotation_bytes(self.d)
        self.struct = _PagedKV()
        ptr = [None if t is None else t.data_ptr() for t in (k_codes, k_norms, v_codes, v_signs, v_norms, v_gammas)]
        _check(lib().tq_paged_kv_init(ctypes.byref(cb_k), ctypes.byref(cb_v), self.d, self.Hkv, self.page_size,
                                      self.num_pages, *ptr, ctypes.byref(self.struct)))
        self.ref = ctypes.byref(self.struct)


def tq_paged_append(kv: PagedKV, k_new, v_new, slots, rot, positions=None, table=None, layout: int = TQ_ROPE_HALF,
                    stream=None):
    """Encodes k_new, v_new [tokens, Hkv, d] (float32 / bfloat16) into slots [tokens] (int64; negative: a padding
    row) of the cache, the keys turned to `positions` (int32) with `table` on the way where they are given."""
    device = kv.device
    if device != _tc.current_device():
        raise ValueError(f"the cache is on device {device}, which is not the current one")
    Hkv, d = kv.Hkv, kv.d
    dtype = k_new.dtype
    if dtype is not _tc.bf16 and dtype is not _tc.f32:
        raise ValueError(f"k_new: dtype {dtype} not float32 / bfloat16")
    tokens = k_new.shape[0]
    strides = []
    for t in (k_new, v_new):
        if t.shape != (tokens, Hkv, d) or t.dtype is not dtype or t.get_device() != device:
            raise ValueError(f"k_new and v_new must be [tokens, {Hkv}, {d}] on device {device}, both of one dtype")
        st, sh, sd = t.stride()
        if sd != 1 or (sh != d and Hkv > 1):
            raise ValueError("k_new and v_new: the heads of a token must be contiguous")
        strides.append(st if tokens > 1 else Hkv * d)            # a single token may have any stride
    at = _in(slots, "slots", device, _tc.i64, tokens)
    pos = tab = None
    n_pos = rot_dim = 0
    if positions is not None and table is not None:
        pos = _in(positions, "positions", device, _tc.i32, tokens)
        tab, n_pos, rot_dim = _table(table, device)
    elif positions is not None or table is not None:
        raise ValueError("positions and table go together")
    _fits(layout)
    status = _lib.tq_paged_append(kv.ref, tokens, k_new.data_ptr(), strides[0], v_new.data_ptr(), strides[1], _tc.code[dtype],
                                  at, pos, tab, n_pos, rot_dim, layout, _prepared(rot, kv), _raw(stream, device))
    if status:
        _check(status)


def _prepared(rot, kv):
    """Address of a rotation prepared for the cache's d, which its size tells."""
    if rot.get_device() != kv.device or rot.dtype is not _tc.u8 or rot.numel() != kv.rot_bytes or not rot.is_contiguous():
        raise ValueError(f"rot must be a rotation prepared for d = {kv.d}: {kv.rot_bytes} contiguous torch.uint8 on device {kv.device}")
    return rot.data_ptr()


def tq_paged_attend_workspace_bytes(kv: PagedKV, B: int, Hq: int, total_q: int, max_q_len: int, max_kv_len: int) -> int:
    _fits(B, Hq, max_q_len)
    _fits(total_q, max_kv_len, bits=64)
    return int(lib().tq_paged_attend_workspace_bytes(kv.ref, B, Hq, total_q, max_q_len, max_kv_len))


def tq_paged_attend(kv: PagedKV, q, q_start, kv_len, page_table, rot, out, max_q_len: int, max_kv_len: int, scale=None,
                    softcap: float = 0.0, window: int = 0, prefix_len=None, slopes=None, ws=None, stream=None):
    """Attention of the newest tokens of B sequences over the paged cache: q [total_q, Hq, d] bfloat16 (token stride
    free), out the same, contiguous; q_start [B + 1], kv_len [B], page_table [B, max_pages], prefix_len [B] int32;
    slopes [Hq] float32."""
    device = kv.device
    if device != _tc.current_device():
        raise ValueError(f"the cache is on device {device}, which is not the current one")
    total_q, Hq, d = shape = q.shape
    if d != kv.d or q.dtype is not _tc.bf16 or q.get_device() != device:
        raise ValueError(f"q must be bfloat16 [total_q, Hq, {kv.d}] on device {device}")
    qt, qh, qd = q.stride()
    if qd != 1 or (qh != d and Hq > 1):
        raise ValueError("q: the heads of a token must be contiguous")
    B = kv_len.shape[0]
    max_pages = page_table.shape[1]
    out_ptr = _in(out, "out", device, _tc.bf16, *shape)
    i32 = _tc.i32
    start = _in(q_start, "q_start", device, i32, B + 1)
    lens = _in(kv_len, "kv_len", device, i32, B)
    pages = _in(page_table, "page_table", device, i32, B, max_pages)
    prefix = None if prefix_len is None else _in(prefix_len, "prefix_len", device, i32, B)
    slope = None if slopes is None else _in(slopes, "slopes", device, _tc.f32, Hq)
    _fits(max_q_len, window)
    _fits(max_kv_len, bits=64)
    if ws is None:
        ws = _empty(max(tq_paged_attend_workspace_bytes(kv, B, Hq, total_q, max_q_len, max_kv_len), 16), _tc.u8,
                    q.device, stream)
    elif ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous and on device {device}")
    status = _lib.tq_paged_attend(kv.ref, B, Hq, total_q, max_q_len, max_kv_len, q.data_ptr(), qt if total_q > 1 else Hq * d,
                                  TQ_BF16, start, lens, pages, max_pages, scale or 0.0, softcap, window, prefix, slope,
                                  _prepared(rot, kv), out_ptr, ws.data_ptr(), ws.nbytes, _raw(stream, device))
    if status:
        _check(status)
    return out


def tq_sync_check(stream=None):
    _check(lib().tq_sync_check(_stream(stream)))


def tq_selftest_wait(limit_ns: int = 1_000_000, stream=None):
    """Enqueue the failure-detection self-test: a bounded device wait that runs out on purpose; the
    next tq_sync_check raises TQError with status TQ_ERR_DEVICE_TIMEOUT once."""
    _check(lib().tq_selftest_wait(int(limit_ns), _stream(stream)))


# ---- allocation helpers (torch device memory) --------------------------------------------------

def empty_mse(n: int, d: int, bits: int, device="cuda"):
    """Output tensors of an Algorithm 1 encode: codes [n, d/32, bits], norms [n]."""
    import torch
    return (torch.empty((n, d // 32, bits), dtype=torch.int32, device=device),
            torch.empty((n,), dtype=torch.float16, device=device))


def empty_prod(n: int, d: int, bits: int, device="cuda"):
    """Outputs of an Algorithm 2 encode at `bits`: codes [n, d/32, bits-1], signs, norms, gammas."""
    import torch
    return (torch.empty((n, d // 32, bits - 1), dtype=torch.int32, device=device),
            torch.empty((n, d // 32), dtype=torch.int32, device=device),
            torch.empty((n,), dtype=torch.float16, device=device),
            torch.empty((n,), dtype=torch.float16, device=device))


def empty_paged(num_pages: int, Hkv: int, page_size: int, d: int, k_bits: int, v_bits: int, v_alg: int = 2, device="cuda"):
    """A PagedKV with new arrays: keys by Algorithm 1 at k_bits, values by Algorithm v_alg at v_bits (Algorithm 2
    with the codebook of v_bits - 1 bits)."""
    import torch
    vb = v_bits - 1 if v_alg == 2 else v_bits
    at = (num_pages, Hkv, page_size)

    def words(*shape):
        return torch.empty((*at, *shape), dtype=torch.int32, device=device)

    def halves():
        return torch.empty(at, dtype=torch.float16, device=device)

    signs = (words(d // 32), halves()) if v_alg == 2 else (None, None)
    return PagedKV(tq_codebook_init(d, k_bits), tq_codebook_init(d, vb), words(d // 32, k_bits), halves(),
                   words(d // 32, vb), halves(), *signs)
