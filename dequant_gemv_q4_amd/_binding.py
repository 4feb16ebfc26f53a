"""ctypes binding of libqgemv (include/qgemv.h): argument marshalling only.

Every function has the name and argument order of its C entry point.  Array arguments may be
torch tensors (their data pointer is passed; device tensors for the compute calls) or plain
integer addresses.  ``stream`` defaults to torch's current HIP stream.  A non-zero status
raises :class:`QgemvError`; nothing is ever computed on the host.  The attention-side calls, which
take several kinds of arrays, check the type, device and layout of the tensors they get (TypeError).
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqgemv.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "qgemv.h")

Q4_0, Q5_0, Q8_0, Q4_K, Q5_K, Q6_K = 2, 6, 8, 12, 13, 14
IQ4_NL, IQ4_XS, Q1_0, AQ4 = 20, 23, 40, 41
F16, BF16 = 1, 30
OP_GEMV, OP_NRM, OP_GUS_NRM, OP_RES, OP_ARGMAX, OP_MOE, OP_NRM_BIAS = range(7)
OP_KV_APPEND, OP_ATTN, OP_ATTN_PROMPT = 7, 8, 9
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_SILU, ACT_GELU_TANH = 0, 1
STATUS = {0: "QG_OK", 1: "QG_ERR_NULL", 2: "QG_ERR_FORMAT", 3: "QG_ERR_SHAPE", 4: "QG_ERR_ALIGN",
          5: "QG_ERR_WORKSPACE", 6: "QG_ERR_LAUNCH", 7: "QG_ERR_ALIAS"}


class QgemvError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({text})")
        self.status = status


_lib = None
_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_SIGS = {
    "qgemv_packed_bytes": (_i64, [_i32, _i64, _i64]),
    "qgemv_pack": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp]),
    "qgemv_pack_codebook": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp]),
    "qgemv_workspace_bytes": (_i64, [_i32, _i32, _i64, _i64, _i32, _i64, _i32]),
    "qgemv": (_i32, [_i32, _vp, _i64, _i64, _vp, _i32, _vp, _vp, _sz, _vp]),
    "qgemv_nrm": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _f32, _i32, _vp, _vp, _sz, _vp]),
    "qgemv_gus_nrm": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _f32, _i32, _vp, _vp, _sz, _vp]),
    "qgemv_nrm_bias": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _f32, _vp, _i32, _vp, _vp, _sz, _vp]),
    "qgemv_gus_act_nrm": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _f32, _i32, _i32, _vp, _vp,
                                 _sz, _vp]),
    "qgemv_qk_norm_rope": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _f32, _vp, _vp,
                                  _vp]),
    "qgemv_res": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _vp, _sz, _vp]),
    "qgemv_argmax": (_i32, [_i32, _vp, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "qgemv_argmax_noalloc": (_i32, [_i32, _vp, _i64, _i64, _vp, _i32, _vp, _vp, _vp]),
    "qgemv_moe": (_i32, [_i32, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp]),
    "qgemm_workspace_bytes": (_i64, [_i32, _i64, _i64, _i64]),
    "qgemm": (_i32, [_i32, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _sz, _vp]),
    "qgemv_moe_error": (_i32, [_vp, _i64, _i64, _i64, _i32, ctypes.POINTER(ctypes.c_int), _vp]),
    "qgemv_attn_workspace_bytes": (_i64, [_i32, _i32, _i32, _i32, _i32]),
    "qgemv_kv_append": (_i32, [_i32, _vp, _vp, _i64, _i32, _i64, _i32, _i32, _vp, _i32, _vp, _vp,
                               _i32, _vp, _vp, _i64, _i64, _vp, _sz, _vp]),
    "qgemv_attn": (_i32, [_i32, _vp, _vp, _i64, _i32, _i64, _i32, _i32, _vp, _i32, _vp, _i32, _vp,
                          _i64, _i32, _f32, _vp, _vp, _sz, _vp]),
    "qgemv_attn_prompt": (_i32, [_i32, _vp, _vp, _i64, _i32, _i64, _i32, _i32, _vp, _i32, _vp, _vp,
                                 _i32, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _sz, _vp]),
    "qgemv_attn_error": (_i32, [_vp, ctypes.POINTER(ctypes.c_int), _vp]),
    "qgemv_route": (_i32, [_vp, _i64, _i32, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _vp,
                           _vp, _vp]),
    "qgemv_status_str": (ctypes.c_char_p, [_i32]),
    "qgemv_layout_version": (_i32, []),
}


def lib():
    """Load libqgemv.so (fails loudly if it was not built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libqgemv.so not built ({LIB_PATH}); run "
                               "`python -m dequant_gemv_q4_amd.build` first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/qgemv.h declares."""
    txt = open(HEADER_PATH).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(qgem[mv][A-Za-z0-9_]*)\s*\(", txt, re.M)


def _p(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(s):
    if s is None:
        # the raw handle: building a Stream object takes 2.7 us, this 0.2
        t = _torch_types()
        return t[4](t[3]())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _nbytes(ws):
    if ws is None:
        return 0
    if isinstance(ws, int):
        raise TypeError("pass ws_bytes together with an integer workspace address")
    return ws.nbytes


def _check(fn, st):
    if st != 0:
        raise QgemvError(fn, st, lib().qgemv_status_str(st).decode())


def qgemv_status_str(status: int) -> str:
    return lib().qgemv_status_str(status).decode()


def qgemv_layout_version() -> int:
    return lib().qgemv_layout_version()


def qgemv_packed_bytes(fmt: int, N: int, K: int) -> int:
    return lib().qgemv_packed_bytes(fmt, N, K)


def qgemv_workspace_bytes(op: int, fmt: int, N: int, K: int, nb: int, n_exp: int = 0,
                          topk: int = 0) -> int:
    return lib().qgemv_workspace_bytes(op, fmt, N, K, nb, n_exp, topk)


def qgemv_pack(fmt, w_gguf, N, K, w_packed, stream=None):
    _check("qgemv_pack", lib().qgemv_pack(fmt, _p(w_gguf), N, K, _p(w_packed), _stream(stream)))


def qgemv_pack_codebook(fmt, w_gguf, N, K, codebook, w_packed, stream=None):
    """codebook: 16 signed bytes on the host (any sequence of ints in [-128, 127]), or None."""
    cb = None
    if codebook is not None:
        vals = [int(v) for v in codebook]
        if len(vals) != 16:
            raise ValueError("the codebook has 16 entries")
        cb = (ctypes.c_int8 * 16)(*vals)
    _check("qgemv_pack_codebook",
           lib().qgemv_pack_codebook(fmt, _p(w_gguf), N, K,
                                     None if cb is None else ctypes.addressof(cb), _p(w_packed),
                                     _stream(stream)))


def qgemv(fmt, W, N, K, x, nb, y, ws=None, ws_bytes=None, stream=None):
    _check("qgemv", lib().qgemv(fmt, _p(W), N, K, _p(x), nb, _p(y), _p(ws),
                                _nbytes(ws) if ws_bytes is None else ws_bytes, _stream(stream)))


def qgemv_nrm(fmt, W, N, K, x, gamma, eps, nb, y, ws=None, ws_bytes=None, stream=None):
    _check("qgemv_nrm", lib().qgemv_nrm(fmt, _p(W), N, K, _p(x), _p(gamma), eps, nb, _p(y), _p(ws),
                                        _nbytes(ws) if ws_bytes is None else ws_bytes,
                                        _stream(stream)))


def qgemv_gus_nrm(fmt, Wg, Wu, N, K, x, gamma, eps, nb, h, ws=None, ws_bytes=None, stream=None):
    _check("qgemv_gus_nrm", lib().qgemv_gus_nrm(fmt, _p(Wg), _p(Wu), N, K, _p(x), _p(gamma), eps,
                                                nb, _p(h), _p(ws),
                                                _nbytes(ws) if ws_bytes is None else ws_bytes,
                                                _stream(stream)))


def qgemv_nrm_bias(fmt, W, N, K, x, gamma, eps, bias, nb, y, ws=None, ws_bytes=None, stream=None):
    _check("qgemv_nrm_bias", lib().qgemv_nrm_bias(fmt, _p(W), N, K, _p(x), _p(gamma), eps, _p(bias),
                                                  nb, _p(y), _p(ws),
                                                  _nbytes(ws) if ws_bytes is None else ws_bytes,
                                                  _stream(stream)))


def qgemv_gus_act_nrm(fmt, Wg, Wu, N, K, x, gamma, eps, act, nb, h, ws=None, ws_bytes=None,
                      stream=None):
    _check("qgemv_gus_act_nrm", lib().qgemv_gus_act_nrm(fmt, _p(Wg), _p(Wu), N, K, _p(x),
                                                        _p(gamma), eps, act, nb, _p(h), _p(ws),
                                                        _nbytes(ws) if ws_bytes is None
                                                        else ws_bytes, _stream(stream)))


def qgemv_qk_norm_rope(qkv, nb, n_q_heads, n_kv_heads, head_dim, rope_half, q_gamma, k_gamma, eps,
                       rope_cos, rope_sin, stream=None):
    _check("qgemv_qk_norm_rope", lib().qgemv_qk_norm_rope(_p(qkv), nb, n_q_heads, n_kv_heads,
                                                          head_dim, rope_half, _p(q_gamma),
                                                          _p(k_gamma), eps, _p(rope_cos),
                                                          _p(rope_sin), _stream(stream)))


def qgemv_res(fmt, W, N, K, x, res, nb, y, ws=None, ws_bytes=None, stream=None):
    _check("qgemv_res", lib().qgemv_res(fmt, _p(W), N, K, _p(x), _p(res), nb, _p(y), _p(ws),
                                        _nbytes(ws) if ws_bytes is None else ws_bytes,
                                        _stream(stream)))


def qgemv_argmax(fmt, W, N, K, x, nb, logits, idx, ws, ws_bytes=None, stream=None):
    _check("qgemv_argmax", lib().qgemv_argmax(fmt, _p(W), N, K, _p(x), nb, _p(logits), _p(idx),
                                              _p(ws), _nbytes(ws) if ws_bytes is None else ws_bytes,
                                              _stream(stream)))


def qgemv_argmax_noalloc(fmt, W, N, K, x, nb, logits, idx, stream=None):
    _check("qgemv_argmax_noalloc", lib().qgemv_argmax_noalloc(fmt, _p(W), N, K, _p(x), nb,
                                                              _p(logits), _p(idx), _stream(stream)))


def qgemv_moe(fmt, W_experts, n_exp, N, K, x, nb, ids, wts, topk, y, ws, ws_bytes=None,
              stream=None):
    _check("qgemv_moe", lib().qgemv_moe(fmt, _p(W_experts), n_exp, N, K, _p(x), nb, _p(ids),
                                        _p(wts), topk, _p(y), _p(ws),
                                        _nbytes(ws) if ws_bytes is None else ws_bytes,
                                        _stream(stream)))


def qgemm_workspace_bytes(fmt: int, N: int, K: int, M: int) -> int:
    return lib().qgemm_workspace_bytes(fmt, N, K, M)


def qgemm(fmt, W, N, K, x, M, y, ws, ws_bytes=None, stream=None):
    _check("qgemm", lib().qgemm(fmt, _p(W), N, K, _p(x), M, _p(y), _p(ws),
                                _nbytes(ws) if ws_bytes is None else ws_bytes, _stream(stream)))


def qgemv_moe_error(ws, n_exp, N, K, fmt, stream=None) -> int:
    flag = ctypes.c_int(0)
    _check("qgemv_moe_error", lib().qgemv_moe_error(_p(ws), n_exp, N, K, fmt, ctypes.byref(flag),
                                                    _stream(stream)))
    return flag.value


def qgemv_attn_workspace_bytes(op: int, n_seq: int, n_q_heads: int, n_kv_heads: int,
                               head_dim: int) -> int:
    return lib().qgemv_attn_workspace_bytes(op, n_seq, n_q_heads, n_kv_heads, head_dim)


# torch's int32, float32, and the cache types by kv_type; the current device's index, its stream
_types = None


def _torch_types():
    global _types
    if _types is None:
        import torch
        _types = (torch.int32, torch.float32, {F16: torch.float16, BF16: torch.bfloat16},
                  torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    return _types


def _t(a, dtype, dev, whole=True):
    """Address of an array of the attention side.  A tensor has to be of the type that the entry
    point reads, on the current device and, unless its rows have a stride argument, contiguous."""
    if a is None or a.__class__ is int:
        return a
    if (dtype is not None and a.dtype is not dtype) or a.get_device() != dev or \
            (whole and not a.is_contiguous()):
        raise TypeError(f"expected a {'contiguous ' if whole else ''}{dtype or 'workspace'} tensor on cuda:{dev}, "
                        f"got {a.dtype}, {a.device}, strides {a.stride()}")
    return a.data_ptr()


def qgemv_kv_append(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                    head_dim, table, max_pages, q_start, kv_len, n_seq, k, v, kv_stride, n_rows, ws,
                    ws_bytes=None, stream=None):
    i32, f32, kv, device, raw = _torch_types()
    d, c = device(), kv.get(kv_type)
    st = lib().qgemv_kv_append(kv_type, _t(k_pages, c, d, False), _t(v_pages, c, d, False), n_pages,
                               page_size, page_stride, n_kv_heads, head_dim, _t(table, i32, d),
                               max_pages, _t(q_start, i32, d), _t(kv_len, i32, d), n_seq,
                               _t(k, f32, d, False), _t(v, f32, d, False), kv_stride, n_rows,
                               _t(ws, None, d), _nbytes(ws) if ws_bytes is None else ws_bytes,
                               raw(d) if stream is None else _stream(stream))
    if st:
        _check("qgemv_kv_append", st)


def qgemv_attn(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads, head_dim,
               table, max_pages, kv_len, n_seq, q, q_stride, n_q_heads, scale, o, ws,
               ws_bytes=None, stream=None):
    i32, f32, kv, device, raw = _torch_types()
    d, c = device(), kv.get(kv_type)
    st = lib().qgemv_attn(kv_type, _t(k_pages, c, d, False), _t(v_pages, c, d, False), n_pages,
                          page_size, page_stride, n_kv_heads, head_dim, _t(table, i32, d), max_pages,
                          _t(kv_len, i32, d), n_seq, _t(q, f32, d, False), q_stride, n_q_heads, scale,
                          _t(o, f32, d), _t(ws, None, d),
                          _nbytes(ws) if ws_bytes is None else ws_bytes,
                          raw(d) if stream is None else _stream(stream))
    if st:
        _check("qgemv_attn", st)


def qgemv_attn_prompt(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                      head_dim, table, max_pages, q_start, kv_len, n_seq, q, q_stride, n_rows,
                      n_q_heads, scale, o, ws, ws_bytes=None, stream=None):
    i32, f32, kv, device, raw = _torch_types()
    d, c = device(), kv.get(kv_type)
    st = lib().qgemv_attn_prompt(kv_type, _t(k_pages, c, d, False), _t(v_pages, c, d, False), n_pages,
                                 page_size, page_stride, n_kv_heads, head_dim, _t(table, i32, d),
                                 max_pages, _t(q_start, i32, d), _t(kv_len, i32, d), n_seq,
                                 _t(q, f32, d, False), q_stride, n_rows, n_q_heads, scale,
                                 _t(o, f32, d), _t(ws, None, d),
                                 _nbytes(ws) if ws_bytes is None else ws_bytes,
                                 raw(d) if stream is None else _stream(stream))
    if st:
        _check("qgemv_attn_prompt", st)


def qgemv_attn_error(ws, stream=None) -> int:
    flag = ctypes.c_int(0)
    _check("qgemv_attn_error", lib().qgemv_attn_error(_p(ws), ctypes.byref(flag), _stream(stream)))
    return flag.value


def qgemv_route(logits, n_rows, n_exp, score, bias, n_group, group_top, topk_group, topk, renorm,
                scale, ids, wts, stream=None):
    i32, f32, _, device, raw = _torch_types()
    d = device()
    st = lib().qgemv_route(_t(logits, f32, d), n_rows, n_exp, score, _t(bias, f32, d), n_group,
                           group_top, topk_group, topk, 1 if renorm else 0, scale, _t(ids, i32, d),
                           _t(wts, f32, d), raw(d) if stream is None else _stream(stream))
    if st:
        _check("qgemv_route", st)
